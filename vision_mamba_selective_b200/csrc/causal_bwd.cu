// causal_bwd.cu -- derivative of the causal selective scan (declared in include/vimscan_causal.h).
//
// With dy = dout silu(z), g_t = C_t dy_t + exp(Delta_(t+1) A) g_(t+1) and
// m_t = exp(Delta_t A) h_(t-1), per token and channel
//
//   dC_t = sum_d dy h_t        dB_t = sum_d g_t Delta u      du = Delta (g . B) + D dy
//   dDelta = sum_n g m A + u (g . B)      ddelta = dDelta sigmoid(delta + bias)
//   dA = sum_t g m Delta       dD = sum_t dy u               dbias = sum_t ddelta
//   dz = dout (C . h + D u) silu'(z)
//
// The sums are fp32: over at most 64 tokens (dA, dD, dbias) or a CTA's channels (dB, dC) in one
// thread or warp, then over the chunks or slices by 16 partial sums or in a row.
//
// Launches: the states every 8 tokens, unless the caller kept them; the adjoint carries
// entering every 64 tokens (both causal_pass); the kernel below over 64-token chunks,
// all independent of one another; the sums over what its CTAs left.  Every sum is taken
// in a fixed order.
#include "causal_kernels.cuh"

#include <algorithm>
#include <cstring>

namespace vimscan {

struct CausalBwdArgs {
    vim_rows u, delta, z, B, C, dout;      // z.data may be null
    vim_rows du, ddelta, dz;
    const float *A, *D, *bias;
    const float *ckpt, *adj;
    float *part_bc;                        // [slices][2][rows][N]: dB then dC of each channel slice
    float *part_a;                         // [chunks][d][N]
    float *part_d;                         // [chunks][2][d]: dD, dbias
    Seqs seqs;
    int64_t rows;                          // batch * L
    int d, chunks_per_row, blocks_per_slice;
};

namespace {

constexpr int kBwdWarps = 4;

// sums v[0 .. n) over the CH channel lanes of a state group (consecutive lanes): lane i < n
// of them, and every lane that equals i modulo n, gets the sum of v[i]
template <int n, int CH>
__device__ __forceinline__ float reduce_channels(float (&v)[n], int cl) {
    float s = reduce_scatter<n, 1>(v, cl);
#pragma unroll
    for (int o = n; o < CH; o <<= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return s;
}

// One CTA: a chunk of 64 tokens and a slice of the channels, 4 warps of CH channels each at a
// time, the chunk's segments of 8 tokens from the last to the first.  Per segment a warp
// runs the recurrence forward from its kept state, holding the decays and m_t in
// registers (one exponential per token, channel and state), then the adjoint backward.
// Bound by latency and issue: 960 instructions per 64 token-channels, 192 of them the packed
// arithmetic, 250 the selects and shuffles of the sums (dB and dC over channels, three
// sums over states), at half an instruction a clock and scheduler.  Two CTAs an SM, with
// room for a segment in registers (at N = 8, whose 16 channels a warp take longer sums, 12 to
// 32 bytes a thread spill all the same): at three the compiler spills 250 bytes a thread (8 x
// 4097 tokens x 384 channels, N = 16, bf16: 308 us; taken at 320 against 510 with the spills, and
// against 330 with m_t in shared memory and loads held back, so that three fit).
template <typename T, int N, int NL, bool PACKED>
__global__ void __launch_bounds__(32 * kBwdWarps, 2) causal_bwd_main(const CausalBwdArgs p) {
    constexpr int LPC = N / NL, CH = 32 / LPC, NP = NL / 2, EPL = kSeg / LPC, NV = 2 * NL;
    __shared__ __align__(16) float Bs[kAdjEvery * N], Cs[kAdjEvery * N];
    __shared__ float acc[kBwdWarps][2][kAdjEvery * N];     // dB, dC
    __shared__ unsigned flags[3][2];                       // tokens of a sequence, its first, its last

    const int w = threadIdx.x / 32, lane = threadIdx.x % 32, q = lane / CH, cl = lane % CH;
    const int b = blockIdx.x / p.chunks_per_row, t0 = (blockIdx.x % p.chunks_per_row) * kAdjEvery;
    const int L = p.seqs.L, slice = blockIdx.y;
    const RowsOf<T> gB(p.B, b, 0), gC(p.C, b, 0);

    unsigned in_lo, in_hi, first_lo = 0, first_hi = 0, last_lo = 0, last_hi = 0;
    if (PACKED) {
        if (w < 2) {
            const int t = t0 + threadIdx.x;
            const int s = sequence_at(p.seqs, t);
            bool in = false, first = false, last = false;
            if (s < p.seqs.n && t < L) {
                in = t >= p.seqs.cu[s];
                first = t == p.seqs.cu[s];
                last = t + 1 == p.seqs.cu[s + 1];
            }
            const unsigned m0 = __ballot_sync(0xffffffffu, in), m1 = __ballot_sync(0xffffffffu, first),
                           m2 = __ballot_sync(0xffffffffu, last);
            if (lane == 0) flags[0][w] = m0, flags[1][w] = m1, flags[2][w] = m2;
        }
        __syncthreads();
        in_lo = flags[0][0], in_hi = flags[0][1];
        first_lo = flags[1][0], first_hi = flags[1][1];
        last_lo = flags[2][0], last_hi = flags[2][1];
    } else {
        const int n = min(L - t0, kAdjEvery);
        in_lo = n >= 32 ? ~0u : (1u << n) - 1;
        in_hi = n >= 64 ? ~0u : n > 32 ? (1u << (n - 32)) - 1 : 0u;
    }
    auto bits = [](unsigned lo, unsigned hi, int seg) { return (seg < 4 ? lo >> (8 * seg) : hi >> (8 * (seg - 4))) & 0xffu; };

    for (int i = threadIdx.x; i < kAdjEvery * N; i += 32 * kBwdWarps) {
        const int r = i / N;
        const bool in = (r < 32 ? in_lo >> r : in_hi >> (r - 32)) & 1u;
        Bs[i] = in ? bits_f32<T>(gB.raw(t0 + r, i % N)) : 0.0f;
        Cs[i] = in ? bits_f32<T>(gC.raw(t0 + r, i % N)) : 0.0f;
    }
#pragma unroll
    for (int i = lane; i < kAdjEvery * N; i += 32) acc[w][0][i] = acc[w][1][i] = 0.0f;
    __syncthreads();

    const bool gate = p.z.data != nullptr;
    const int cblocks = (p.d + CH * kBwdWarps - 1) / (CH * kBwdWarps);
    const int cb0 = slice * p.blocks_per_slice, cb1 = min(cb0 + p.blocks_per_slice, cblocks);
    const int64_t kept_row = (int64_t)b * ((L + kCkEvery - 1) / kCkEvery) + t0 / kCkEvery;
    const int64_t chunk = blockIdx.x;
    const int last_kept = (min(L - t0, kAdjEvery) - 1) / kSeg;

#pragma unroll 1
    for (int cb = cb0; cb < cb1; ++cb) {
        const int c_at = (cb * kBwdWarps + w) * CH + cl;
        const bool live = c_at < p.d;
        const int c = live ? c_at : p.d - 1;
        const RowsOf<T> gu(p.u, b, c), gd(p.delta, b, c), gz(gate ? p.z : p.u, b, c), go(p.dout, b, c);
        const RowsOf<T> pu(p.du, b, c), pd(p.ddelta, b, c), pz(gate ? p.dz : p.du, b, c);
        float2 A2[NP], dA[NP], g[NP];
        load_row<NP>(p.A + (int64_t)c * N + q * NL, A2);
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            A2[i] = decay_rate(A2[i]);
            dA[i] = g[i] = f2(0.0f, 0.0f);
        }
        const float bias = p.bias[c], Dc = p.D[c];
        float dD = 0.0f, dbias = 0.0f;
        // the carry entering the chunk from behind, where its last token's sequence goes on
        const bool goes_on = PACKED ? (in_hi >> 31) && !(last_hi >> 31) : t0 + kAdjEvery < L;
        if (goes_on) load_row<NP>(p.adj + (chunk * p.d + c) * N + q * NL, g);

        const int top = last_kept;
        uint32_t ru[EPL], rd[EPL], rz[EPL], ro[EPL];
        float2 hk[NP];
        auto fetch = [&](int seg) {
#pragma unroll
            for (int e = 0; e < EPL; ++e) {
                // past the row's end its last token is read, and dropped
                const int t = min(t0 + seg * kSeg + e * LPC + q, L - 1);
                ru[e] = gu.raw(t), rd[e] = gd.raw(t), rz[e] = gz.raw(t), ro[e] = go.raw(t);
            }
            // (where no sequence enters a segment nothing was kept; its first token resets)
            load_row<NP>(p.ckpt + ((kept_row + min(seg, last_kept)) * p.d + c) * N + q * NL, hk);
        };
        fetch(top);
#pragma unroll 1
        for (int seg = top; seg >= 0; --seg) {
            const unsigned in = bits(in_lo, in_hi, seg);
            const unsigned first = PACKED ? bits(first_lo, first_hi, seg) : 0u;
            const unsigned last = PACKED ? bits(last_lo, last_hi, seg) : 0u;
            // the lane's tokens
            float u[EPL], dt[EPL], x[EPL], dy[EPL], slope[EPL], dgate[EPL];
#pragma unroll
            for (int e = 0; e < EPL; ++e) {
                // lanes past d run the last channel with nothing flowing in: their sums are zero
                const bool ok = live && (in >> (e * LPC + q) & 1u);
                u[e] = bits_f32<T>(ru[e]);
                const float z = bits_f32<T>(rz[e]), o = bits_f32<T>(ro[e]);
                dt[e] = ok ? softplus_slope(bits_f32<T>(rd[e]) + bias, slope[e]) : 0.0f;
                const float sg = sigmoid(z);
                x[e] = ok ? dt[e] * u[e] : 0.0f;
                dy[e] = ok ? (gate ? o * (z * sg) : o) : 0.0f;
                dgate[e] = o * (sg * fmaf(z, 1.0f - sg, 1.0f));
            }
            float2 h[NP];
#pragma unroll
            for (int i = 0; i < NP; ++i) h[i] = hk[i];
            if (seg > 0) fetch(seg - 1);

            // where the lane adds its sum over channels of token pair (r, r + 1)
            auto slot = [&](int which, int r) {
                return &acc[w][which][(r + (cl % NV) / NL) * N + q * NL + cl % NL];
            };

            // forward: a_t, m_t, C . h and the terms of dC
            float2 a[kSeg][NP], m[kSeg][NP];
            float y[EPL], part[LPC], v[NV];
#pragma unroll
            for (int j = 0; j < kSeg; ++j) {
                const int e = j / LPC, l = j % LPC, r = seg * kSeg + j;
                const float dtj = __shfl_sync(0xffffffffu, dt[e], l * CH + cl);
                const float xj = __shfl_sync(0xffffffffu, x[e], l * CH + cl);
                const float dyj = __shfl_sync(0xffffffffu, dy[e], l * CH + cl);
                float2 rb[NP], rc[NP], s;
                load_row<NP>(&Bs[r * N + q * NL], rb);
                load_row<NP>(&Cs[r * N + q * NL], rc);
                const bool reset = PACKED && ((first >> j & 1u) || !(in >> j & 1u));
#pragma unroll
                for (int i = 0; i < NP; ++i) {
                    a[j][i] = decay(A2[i], dtj);
                    m[j][i] = mul2(a[j][i], h[i]);
                    if (reset) m[j][i] = f2(0.0f, 0.0f);
                    h[i] = fma2(rb[i], f2(xj, xj), m[j][i]);
                    s = i == 0 ? mul2(rc[i], h[i]) : fma2(rc[i], h[i], s);
                    const float2 k = mul2(h[i], f2(dyj, dyj));
                    v[j % 2 * NL + 2 * i] = k.x;
                    v[j % 2 * NL + 2 * i + 1] = k.y;
                }
                part[l] = s.x + s.y;
                if (l == LPC - 1) y[e] = reduce_scatter<LPC, CH>(part, q);
                if (j % 2) {
                    const float sum = reduce_channels<NV, CH>(v, cl);
                    if (NV >= CH || cl < NV) *slot(1, r - 1) += sum;
                }
            }

            // backward: g_t and everything that follows from it
            float gb[EPL], ga[EPL], part2[LPC];
#pragma unroll
            for (int j = kSeg - 1; j >= 0; --j) {
                const int e = j / LPC, l = j % LPC, r = seg * kSeg + j;
                const float dtj = __shfl_sync(0xffffffffu, dt[e], l * CH + cl);
                const float xj = __shfl_sync(0xffffffffu, x[e], l * CH + cl);
                const float dyj = __shfl_sync(0xffffffffu, dy[e], l * CH + cl);
                float2 rb[NP], rc[NP], sb, sa;
                load_row<NP>(&Bs[r * N + q * NL], rb);
                load_row<NP>(&Cs[r * N + q * NL], rc);
                const bool cut = PACKED && ((last >> j & 1u) || !(in >> j & 1u));
#pragma unroll
                for (int i = 0; i < NP; ++i) {
                    if (cut) g[i] = f2(0.0f, 0.0f);
                    g[i] = fma2(rc[i], f2(dyj, dyj), g[i]);
                    sb = i == 0 ? mul2(g[i], rb[i]) : fma2(g[i], rb[i], sb);
                    const float2 k = mul2(g[i], f2(xj, xj));
                    v[j % 2 * NL + 2 * i] = k.x;
                    v[j % 2 * NL + 2 * i + 1] = k.y;
                    const float2 gm = mul2(g[i], m[j][i]);
                    dA[i] = fma2(gm, f2(dtj, dtj), dA[i]);
                    sa = i == 0 ? mul2(gm, A2[i]) : fma2(gm, A2[i], sa);
                    g[i] = mul2(a[j][i], g[i]);
                }
                part[l] = sb.x + sb.y;
                part2[l] = sa.x + sa.y;
                if (l == 0) {
                    gb[e] = reduce_scatter<LPC, CH>(part, q);
                    ga[e] = reduce_scatter<LPC, CH>(part2, q);
                }
                if (j % 2 == 0) {
                    const float sum = reduce_channels<NV, CH>(v, cl);
                    if (NV >= CH || cl < NV) *slot(0, r) += sum;
                }
            }

#pragma unroll
            for (int e = 0; e < EPL; ++e) {
                const int r = e * LPC + q, t = t0 + seg * kSeg + r;
                const float ddt = fmaf(ga[e], kLn2, u[e] * gb[e]) * slope[e];
                if (live && (in >> r & 1u)) {
                    pu.put(t, fmaf(dt[e], gb[e], Dc * dy[e]));
                    pd.put(t, ddt);
                    if (gate) pz.put(t, dgate[e] * fmaf(Dc, u[e], y[e]));
                    dD = fmaf(dy[e], u[e], dD);
                    dbias += ddt;
                }
            }
        }
        if (live) store_row<NP>(p.part_a + (chunk * p.d + c) * N + q * NL, dA);
#pragma unroll
        for (int o = CH; o < 32; o <<= 1) {
            dD += __shfl_xor_sync(0xffffffffu, dD, o);
            dbias += __shfl_xor_sync(0xffffffffu, dbias, o);
        }
        if (live && q == 0) {
            p.part_d[(2 * chunk) * p.d + c] = dD;
            p.part_d[(2 * chunk + 1) * p.d + c] = dbias;
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * kAdjEvery * N; i += 32 * kBwdWarps) {
        const int which = i / (kAdjEvery * N), k = i % (kAdjEvery * N), r = k / N;
        if (!((r < 32 ? in_lo >> r : in_hi >> (r - 32)) & 1u)) continue;
        float s = 0.0f;
#pragma unroll
        for (int x = 0; x < kBwdWarps; ++x) s += acc[x][which][k];
        p.part_bc[((int64_t)(slice * 2 + which) * p.rows + (int64_t)b * L + t0 + r) * N + k % N] = s;
    }
}

// The sums over what causal_bwd_main's CTAs left, in one launch: the first `param_ctas` CTAs add up
// dA, dD and dbias over the chunks (16 partial sums per element joined in shared memory), the
// others dB and dC over the channel slices.
struct CausalSumArgs {
    const float *part_bc, *part_a, *part_d;
    float *dB, *dC, *dA, *dD, *dbias;
    const int *cu;
    int n_seqs, slices, chunks, d, N, param_ctas;
    int64_t rows;
};
constexpr int kSumX = 32, kSumY = 16, kSumThreads = kSumX * kSumY;
__global__ void __launch_bounds__(kSumThreads) causal_bwd_sums(const CausalSumArgs p) {
    __shared__ float part[kSumY][kSumX];
    if ((int)blockIdx.x >= p.param_ctas) {
        const int64_t n = p.rows * p.N, i = (int64_t)(blockIdx.x - p.param_ctas) * kSumThreads + threadIdx.x;
        if (i >= 2 * n) return;
        const int which = i >= n;
        const int64_t k = which ? i - n : i;
        if (p.cu) {                                        // tokens of no sequence keep what they held
            const int64_t t = k / p.N;
            if (t < max(p.cu[0], 0) || t >= p.cu[p.n_seqs]) return;
        }
        float s = 0.0f;
        for (int x = 0; x < p.slices; ++x) s += p.part_bc[(x * 2 + which) * n + k];
        (which ? p.dC : p.dB)[k] = s;
        return;
    }
    const int tx = threadIdx.x % kSumX, ty = threadIdx.x / kSumX;
    const int64_t na = (int64_t)p.d * p.N, n = na + 2 * (int64_t)p.d;
    const int64_t i = (int64_t)blockIdx.x * kSumX + tx;
    const float *src = i < na ? p.part_a + i : p.part_d + (i - na);
    const int64_t step = i < na ? na : 2 * (int64_t)p.d;
    float s = 0.0f;
    if (i < n)
        for (int k = ty; k < p.chunks; k += kSumY) s += src[k * step];
    part[ty][tx] = s;
    __syncthreads();
    if (ty == 0 && i < n) {
        s = 0.0f;
#pragma unroll
        for (int y = 0; y < kSumY; ++y) s += part[y][tx];
        if (i < na) p.dA[i] = s;
        else if (i < na + p.d) p.dD[i - na] = s;
        else p.dbias[i - na - p.d] = s;
    }
}

// ----------------------------------------------------------------------------
// plan of a call: chunks, channel slices and the workspace
// ----------------------------------------------------------------------------
struct CausalBwdPlan {
    int64_t chunks;
    int chunks_per_row, slices, blocks_per_slice;
    size_t o_ckpt, o_adj, o_bc, o_a, o_d, total;
};

CausalBwdPlan causal_bwd_plan(int batch, int L, int d, int N, bool has_ckpt) {
    CausalBwdPlan pl;
    std::memset(&pl, 0, sizeof(pl));
    pl.chunks_per_row = (L + kAdjEvery - 1) / kAdjEvery;
    pl.chunks = (int64_t)batch * pl.chunks_per_row;
    const int ch = N == 16 ? 8 : N == 2 ? 32 : 16;
    const int blocks = (d + ch * kBwdWarps - 1) / (ch * kBwdWarps);
    // enough CTAs for two rounds on every SM, two at a time there; more slices only cost
    // traffic (each leaves 2 N sums per token)
    const int64_t want = 148 * 2 * 2;
    const int64_t s = std::max<int64_t>(1, std::min<int64_t>(blocks, (want + pl.chunks - 1) / std::max<int64_t>(pl.chunks, 1)));
    pl.blocks_per_slice = (int)((blocks + s - 1) / s);
    pl.slices = (blocks + pl.blocks_per_slice - 1) / pl.blocks_per_slice;
    size_t o = 0;
    auto take = [&](size_t floats) { const size_t at = o; o += round_up(floats * sizeof(float)); return at; };
    pl.o_ckpt = take(has_ckpt ? 0 : (size_t)batch * ((L + kCkEvery - 1) / kCkEvery) * d * N);
    pl.o_adj = take((size_t)pl.chunks * d * N);
    pl.o_bc = take((size_t)pl.slices * 2 * batch * L * N);
    pl.o_a = take((size_t)pl.chunks * d * N);
    pl.o_d = take((size_t)pl.chunks * 2 * d);
    pl.total = o;
    return pl;
}

template <typename T, int N, int NL>
vim_status launch_main(const CausalBwdArgs &a, const CausalBwdPlan &pl, cudaStream_t stream) {
    auto kernel = a.seqs.cu ? causal_bwd_main<T, N, NL, true> : causal_bwd_main<T, N, NL, false>;
    kernel<<<dim3((unsigned)pl.chunks, pl.slices), 32 * kBwdWarps, 0, stream>>>(a);
    return cudaGetLastError() == cudaSuccess ? VIM_OK : VIM_ERR_CUDA;
}

}  // namespace
}  // namespace vimscan

using namespace vimscan;

extern "C" {

size_t causal_bwd_workspace_bytes(int batch, int L, int d_inner, int d_state, int has_ckpt) {
    if (batch <= 0 || L <= 0 || d_inner <= 0 || !supported_state(d_state)) return 0;
    return causal_bwd_plan(batch, L, d_inner, d_state, has_ckpt != 0).total;
}

vim_status causal_scan_bwd(const vim_scan_bwd_io *io, const float *A, const float *D, const float *delta_bias,
                           float *dB, float *dC, float *dA, float *dD, float *ddelta_bias, int batch, int L,
                           int d_inner, int d_state, vim_dtype dt, const int32_t *cu_seqlens, int n_seqs,
                           const float *ckpt, void *workspace, size_t workspace_bytes, cudaStream_t stream) {
    if (!io) return VIM_ERR_INVALID_ARG;
    const vim_rows &u = io->u, &delta = io->delta, &z = io->z, &B = io->B, &C = io->C, &dout = io->dout,
                   &du = io->du, &ddelta = io->ddelta, &dz = io->dz;
    vim_status st = check_sizes(batch, L, d_inner, dt);
    if (st != VIM_OK) return st;
    if (!supported_state(d_state)) return VIM_ERR_UNSUPPORTED;
    vim_sequences seqs;
    std::memset(&seqs, 0, sizeof(seqs));
    seqs.cu_seqlens = cu_seqlens;
    seqs.n_seqs = cu_seqlens ? n_seqs : batch;
    CausalArgs pass;
    std::memset(&pass, 0, sizeof(pass));
    st = make_seqs(&seqs, batch, L, 16, 0, &pass.seqs);
    if (st != VIM_OK) return st;
    if (d_inner == 0) return VIM_OK;
    if (!dA || !dD || !ddelta_bias || misaligned(dA, 4) || misaligned(dD, 4) || misaligned(ddelta_bias, 4))
        return VIM_ERR_INVALID_ARG;
    if (batch == 0 || L == 0 || pass.seqs.n == 0) {        // no token: the parameters' derivatives are zero
        const size_t n = (size_t)d_inner * sizeof(float);
        const bool ok = cudaMemsetAsync(dA, 0, n * d_state, stream) == cudaSuccess &&
                        cudaMemsetAsync(dD, 0, n, stream) == cudaSuccess &&
                        cudaMemsetAsync(ddelta_bias, 0, n, stream) == cudaSuccess;
        return ok ? VIM_OK : VIM_ERR_CUDA;
    }
    if (bad_rows(u, dt) || bad_rows(delta, dt) || bad_rows(B, dt) || bad_rows(C, dt) || bad_rows(dout, dt) ||
        (z.data && bad_rows(z, dt)))
        return VIM_ERR_INVALID_ARG;
    if (bad_params(A, D, delta_bias)) return VIM_ERR_INVALID_ARG;
    if (bad_out(du, dt, batch, L, d_inner) || bad_out(ddelta, dt, batch, L, d_inner)) return VIM_ERR_INVALID_ARG;
    if (!z.data != !dz.data || (z.data && bad_out(dz, dt, batch, L, d_inner))) return VIM_ERR_INVALID_ARG;
    // an output over an input (other warps may still have to read it), or over another output
    const vim_rows *outs[] = {&du, &ddelta, &dz};
    for (int k = 0; k < 3; ++k) {
        for (const vim_rows *i : {&u, &delta, &z, &dout})
            if (rows_meet(*outs[k], d_inner, *i, d_inner, dt, batch, L)) return VIM_ERR_INVALID_ARG;
        for (const vim_rows *i : {&B, &C})
            if (rows_meet(*outs[k], d_inner, *i, d_state, dt, batch, L)) return VIM_ERR_INVALID_ARG;
        for (int j = 0; j < k; ++j)
            if (rows_meet(*outs[k], d_inner, *outs[j], d_inner, dt, batch, L)) return VIM_ERR_INVALID_ARG;
    }
    if (!dB || !dC || misaligned(dB, 4) || misaligned(dC, 4) || misaligned(ckpt, 16)) return VIM_ERR_INVALID_ARG;
    const CausalBwdPlan pl = causal_bwd_plan(batch, L, d_inner, d_state, ckpt != nullptr);
    if (pl.chunks > INT32_MAX || pl.slices > 65535) return VIM_ERR_UNSUPPORTED;
    if (!workspace || workspace_bytes < pl.total || misaligned(workspace, kAlign)) return VIM_ERR_WORKSPACE;
    char *ws = static_cast<char *>(workspace);
    auto at = [&](size_t o) { return reinterpret_cast<float *>(ws + o); };

    pass.u = u, pass.delta = delta, pass.z = z, pass.B = B, pass.C = C, pass.dout = dout;
    pass.A = A, pass.D = D, pass.bias = delta_bias;
    pass.d = d_inner;
    pass.vec_bc = row_vectors(B, dt, batch, L, lane_states(d_state)) && row_vectors(C, dt, batch, L, lane_states(d_state));
    if (!ckpt) {
        pass.ckpt = at(pl.o_ckpt);
        st = launch_pass<kStates>(pass, d_state, dt, stream);
        if (st != VIM_OK) return st;
        ckpt = pass.ckpt;
    }
    pass.ckpt = nullptr;
    pass.adj = at(pl.o_adj);
    st = launch_pass<kAdjoint>(pass, d_state, dt, stream);
    if (st != VIM_OK) return st;

    CausalBwdArgs a;
    std::memset(&a, 0, sizeof(a));
    a.u = u, a.delta = delta, a.z = z, a.B = B, a.C = C, a.dout = dout;
    a.du = du, a.ddelta = ddelta, a.dz = dz;
    a.A = A, a.D = D, a.bias = delta_bias;
    a.ckpt = ckpt, a.adj = pass.adj;
    a.part_bc = at(pl.o_bc), a.part_a = at(pl.o_a), a.part_d = at(pl.o_d);
    a.seqs = pass.seqs;
    a.rows = (int64_t)batch * L;
    a.d = d_inner, a.chunks_per_row = pl.chunks_per_row, a.blocks_per_slice = pl.blocks_per_slice;
    const bool f = dt == VIM_F32;
    switch (d_state) {
        case 2: st = f ? launch_main<float, 2, 2>(a, pl, stream) : launch_main<__nv_bfloat16, 2, 2>(a, pl, stream); break;
        case 4: st = f ? launch_main<float, 4, 2>(a, pl, stream) : launch_main<__nv_bfloat16, 4, 2>(a, pl, stream); break;
        case 8: st = f ? launch_main<float, 8, 4>(a, pl, stream) : launch_main<__nv_bfloat16, 8, 4>(a, pl, stream); break;
        default: st = f ? launch_main<float, 16, 4>(a, pl, stream) : launch_main<__nv_bfloat16, 16, 4>(a, pl, stream);
    }
    if (st != VIM_OK) return st;

    const int64_t n_bc = 2 * a.rows * d_state, n_par = (int64_t)d_inner * (d_state + 2);
    const int64_t param_ctas = (n_par + kSumX - 1) / kSumX, bc_ctas = (n_bc + kSumThreads - 1) / kSumThreads;
    if (param_ctas + bc_ctas > INT32_MAX) return VIM_ERR_UNSUPPORTED;
    CausalSumArgs sum = {a.part_bc, a.part_a, a.part_d, dB, dC, dA, dD, ddelta_bias, cu_seqlens, n_seqs, pl.slices,
                         (int)pl.chunks, d_inner, d_state, (int)param_ctas, a.rows};
    causal_bwd_sums<<<(unsigned)(param_ctas + bc_ctas), kSumThreads, 0, stream>>>(sum);
    return cudaGetLastError() == cudaSuccess ? VIM_OK : VIM_ERR_CUDA;
}

}  // extern "C"
