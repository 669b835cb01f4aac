// causal_kernels.cuh -- sm_100a kernels of the causal selective scan over whole sequences.
//
//   Delta_t = softplus(delta_t + bias);   h_t = exp(Delta_t A) h_(t-1) + Delta_t B_t u_t
//   y_t     = (C_t . h_t + D u_t) silu(z_t)
//
// and, with time reversed, the adjoint of h that its derivative needs:
//
//   g_t = C_t dy_t + carry_t,  carry_(t-1) = exp(Delta_t A) g_t,  dy_t = dout_t silu(z_t).
//
// What bounds it: A is free per channel and state, so every token-channel takes N
// exponentials, and the special-function unit gives 16 a clock and SM: with softplus and
// the gate's sigmoid 20 for N = 16, 1.25 clocks a token-channel, against 0.2 clocks of
// memory traffic at bf16 and 0.5 of packed FP32 work.  Cutting the sequence into chunks
// that run side by side costs a second pass over those exponentials (a chunk's end state
// first, then its outputs), so a sequence is walked once, by one CTA per few channels,
// and the parallelism comes from the states instead: the N states of a channel are
// spread over N / NL neighbouring lanes, NL states (1 to 4, in f32x2 pairs) a lane.  The
// fewer channels there are, the thinner they are spread (see causal_lanes()).
//
// A warp handles 32 / LPC channels, LPC = N / NL, in groups of LPC tokens:
//   - each lane forms Delta and Delta u of ONE token of the group for its channel, a group
//     ahead, and leaves them in a ring of shared memory that only its warp reads: no
//     transcendental is computed twice, and no CTA barrier stands in the token loop;
//   - the recurrence runs token by token on the lane's states, giving LPC partial sums of
//     C . h, which one reduce-scatter over the channel's lanes turns into the y of the
//     lane's own token; the same lane gates it and puts it where it had read u.
// u, delta and z arrive by cp.async in tiles of kTok tokens, two tiles deep; B and C pass
// through registers, a tile ahead, and stand in shared memory in fp32.  Tiles and groups
// are aligned to the token axis, and tokens outside the sequence get Delta = 0 and
// Delta u = 0, which leave the state as it is.
#pragma once

#include "causal.cuh"

namespace vimscan {

struct CausalArgs {
    vim_rows u, delta, z, B, C;     // z.data may be null
    vim_rows dout;                  // adjoint only
    vim_rows y;
    const float *A, *D, *bias;      // [d][N], [d], [d]
    Seqs seqs;                      // seqs.cu null: one sequence per batch row
    const float *state;             // [n_slots][d][N] or null: initial states
    float *state_out;               // [n_slots][d][N] or null: final states
    float *ckpt;                    // [batch][ceil(L / kCkEvery)][d][N] or null
    float *adj;                     // adjoint: carries, [batch][ceil(L / kAdjEvery)][d][N]
    int d;
    int vec_act, vec_bc;            // rows of u, delta, z, y (B, C) move as 16-byte vectors
};
constexpr int kCkEvery = 8;         // tokens between kept states
constexpr int kAdjEvery = 64;       // tokens between kept adjoint carries

enum CausalMode {
    kForward = 0,                   // y, and where asked for final states and kept states
    kStates = 1,                    // kept states only
    kAdjoint = 2                    // adjoint carries
};

namespace {

constexpr int kPassThreads = 128;

// sums p[0 .. n) over the n neighbouring lanes of a group: lane i of it gets the sum of
// p[i].  Each step halves the values a lane holds.
template <int n>
__device__ __forceinline__ float reduce_scatter(float (&p)[n], int lane) {
#pragma unroll
    for (int half = n / 2; half >= 1; half >>= 1) {
        const bool upper = lane & half;
#pragma unroll
        for (int i = 0; i < half; ++i) {
            const float send = upper ? p[i] : p[i + half];
            const float keep = upper ? p[i + half] : p[i];
            p[i] = keep + __shfl_xor_sync(0xffffffffu, send, half);
        }
    }
    return p[0];
}

// shared memory of causal_pass
template <typename T, int N, int NL, int TOK>
struct PassStage {
    static constexpr int kLanes = N / NL;                  // lanes per channel
    static constexpr int kCh = kPassThreads / kLanes;      // channels per CTA
    static constexpr int kRaw = TOK * kCh;                 // elements of one raw tile
    static constexpr int kBcRow = NL == 1 ? TOK + 4 : N;   // fp32 B/C: [n][tok] or [tok][n]
    static constexpr int kBc = NL == 1 ? N * kBcRow : TOK * N;
    // ring rows: kLanes (Delta, Delta u) pairs and 16 bytes, so that the 16-byte reads of a
    // warp's channels fall into different banks
    static constexpr int kRingRow = kLanes * 2 + 4;
    static constexpr int kRing = (kPassThreads / kLanes) * kRingRow;
    T raw[2][3][kRaw];                                     // u (then y) or dout, delta, z
    float bc[2][2][kBc];
    float ring[2][kRing];
};

template <typename T, int N, int NL, int TOK, int MODE>
__global__ void __launch_bounds__(kPassThreads) causal_pass(const CausalArgs p) {
    using S = PassStage<T, N, NL, TOK>;
    constexpr int LPC = S::kLanes, CH = S::kCh, V = Vec<T>::n;
    constexpr int NP = NL / 2;                             // f32x2 pairs per lane (NL > 1)
    extern __shared__ __align__(16) unsigned char smem_raw[];
    S &sm = *reinterpret_cast<S *>(smem_raw);

    const int blocks = (p.d + CH - 1) / CH;
    const int s = blockIdx.x / blocks, c0 = (blockIdx.x % blocks) * CH;
    const Seq seq = sequence(p.seqs, s);
    const int64_t b = p.seqs.cu ? 0 : s;
    const int tid = threadIdx.x, q = tid % LPC, cl = tid / LPC, c = c0 + cl;
    const bool live = c < p.d;
    if (seq.slot < 0) return;                              // a padding entry

    const T *gu = static_cast<const T *>((MODE == kAdjoint ? p.dout : p.u).data) +
                  b * (MODE == kAdjoint ? p.dout : p.u).batch_stride + c0;
    const T *gd = static_cast<const T *>(p.delta.data) + b * p.delta.batch_stride + c0;
    const T *gz = p.z.data ? static_cast<const T *>(p.z.data) + b * p.z.batch_stride + c0 : nullptr;
    const T *gB = static_cast<const T *>(p.B.data) + b * p.B.batch_stride;
    const T *gC = static_cast<const T *>(p.C.data) + b * p.C.batch_stride;
    T *gy = static_cast<T *>(const_cast<void *>(p.y.data)) + b * p.y.batch_stride + c0;
    const int64_t ru = (MODE == kAdjoint ? p.dout : p.u).row_stride;

    // the lane's parameters and state; channels past d run on zeros
    float A2[NL], h[NL], Dc = 0.0f, bias = 0.0f;
#pragma unroll
    for (int i = 0; i < NL; ++i) {
        A2[i] = live ? p.A[(int64_t)c * N + q * NL + i] * kLog2e : 0.0f;
        h[i] = 0.0f;
    }
    if (live) {
        bias = p.bias[c];
        if (MODE == kForward) Dc = p.D[c];
        if (p.state && !seq.fresh) {
            const float *from = p.state + (seq.slot * p.d + c) * N + q * NL;
#pragma unroll
            for (int i = 0; i < NL; ++i) h[i] = from[i];
        }
    }

    const int first = seq.start / TOK;                     // tiles first .. last - 1 of the token axis
    const int tiles = seq.end > seq.start ? (seq.end + TOK - 1) / TOK - first : 0;
    auto tile_at = [&](int k) { return (MODE == kAdjoint ? first + tiles - 1 - k : first + k) * TOK; };

    // raw tile k -> buffer k & 1 (rows outside the sequence are not read)
    auto load_tile = [&](int k) {
        const int t0 = tile_at(k);
        T *dst = &sm.raw[k & 1][0][0];
        if (p.vec_act) {
            constexpr int PER = CH / V > 0 ? CH / V : 1;   // vectors per row
#pragma unroll 1
            for (int i = tid; i < TOK * PER; i += kPassThreads) {
                const int r = i / PER, j = (i % PER) * V, t = t0 + r;
                if (t < seq.start || t >= seq.end || c0 + j >= p.d) continue;
                T *at = dst + r * CH + j;
                cp_async16(at, gu + t * ru + j, true);
                cp_async16(at + S::kRaw, gd + t * p.delta.row_stride + j, true);
                if (gz && MODE != kStates) cp_async16(at + 2 * S::kRaw, gz + t * p.z.row_stride + j, true);
            }
            cp_async_commit();
        } else {
#pragma unroll 1
            for (int i = tid; i < TOK * CH; i += kPassThreads) {
                const int r = i / CH, j = i % CH, t = t0 + r;
                if (t < seq.start || t >= seq.end || c0 + j >= p.d) continue;
                dst[i] = gu[t * ru + j];
                dst[S::kRaw + i] = gd[t * p.delta.row_stride + j];
                if (gz && MODE != kStates) dst[2 * S::kRaw + i] = gz[t * p.z.row_stride + j];
            }
        }
    };

    // B (not for the adjoint) and C (not for kept states alone) of a tile, as vectors of V
    // consecutive (token, state) values in registers; zeros outside the sequence, so that
    // Delta u = 0 meets no NaN there
    constexpr bool HAS_B = MODE != kAdjoint, HAS_C = MODE != kStates;
    constexpr int BCV = TOK * N / V;                       // vectors of one of them
    constexpr int PF = (BCV + kPassThreads - 1) / kPassThreads;
    uint4 pre[2][PF];
    auto load_bc = [&](int k) {
        const int t0 = tile_at(k);
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            if (w == 0 ? !HAS_B : !HAS_C) continue;
            const T *src = w == 0 ? gB : gC;
            const int64_t row = w == 0 ? p.B.row_stride : p.C.row_stride;
#pragma unroll
            for (int f = 0; f < PF; ++f) {
                const int v = tid + f * kPassThreads;
                pre[w][f] = make_uint4(0, 0, 0, 0);
                if (v >= BCV) continue;
                if (N % V == 0 && p.vec_bc) {
                    const int t = t0 + v * V / N;
                    if (t >= seq.start && t < seq.end)
                        pre[w][f] = *reinterpret_cast<const uint4 *>(src + t * row + v * V % N);
                } else {
                    T e[V];
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        const int t = t0 + (v * V + i) / N;
                        e[i] = t >= seq.start && t < seq.end ? src[t * row + (v * V + i) % N] : from_f32<T>(0.0f);
                    }
                    pre[w][f] = *reinterpret_cast<const uint4 *>(e);
                }
            }
        }
    };
    auto store_bc = [&](int k) {
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            if (w == 0 ? !HAS_B : !HAS_C) continue;
#pragma unroll
            for (int f = 0; f < PF; ++f) {
                const int v = tid + f * kPassThreads;
                if (v >= BCV) continue;
                float e[V];
                unpack16(pre[w][f], e);
                float *dst = sm.bc[k & 1][w];
                if constexpr (NL == 1) {
#pragma unroll
                    for (int i = 0; i < V; ++i) dst[((v * V + i) % N) * S::kBcRow + (v * V + i) / N] = e[i];
                } else {
#pragma unroll
                    for (int i = 0; i < V; i += 4)
                        *reinterpret_cast<float4 *>(dst + v * V + i) = make_float4(e[i], e[i + 1], e[i + 2], e[i + 3]);
                }
            }
        }
    };

    // rows of y that the last tile left in its raw buffer -> global
    auto store_tile = [&](int k) {
        const int t0 = tile_at(k);
        const T *src = &sm.raw[k & 1][0][0];
        if (p.vec_act) {
            constexpr int PER = CH / V > 0 ? CH / V : 1;
#pragma unroll 1
            for (int i = tid; i < TOK * PER; i += kPassThreads) {
                const int r = i / PER, j = (i % PER) * V, t = t0 + r;
                if (t < seq.start || t >= seq.end || c0 + j >= p.d) continue;
                *reinterpret_cast<uint4 *>(gy + t * p.y.row_stride + j) = *reinterpret_cast<const uint4 *>(src + r * CH + j);
            }
        } else {
#pragma unroll 1
            for (int i = tid; i < TOK * CH; i += kPassThreads) {
                const int r = i / CH, j = i % CH, t = t0 + r;
                if (t < seq.start || t >= seq.end || c0 + j >= p.d) continue;
                gy[t * p.y.row_stride + j] = src[i];
            }
        }
    };

    constexpr int GROUPS = TOK / LPC;
    if (tiles > 0) {
        load_tile(0);
        load_bc(0);
        store_bc(0);
    }
#pragma unroll 1
    for (int k = 0; k < tiles; ++k) {
        cp_async_wait_all();
        __syncthreads();                                   // tile k is there; tile k - 1 is done with
        if (MODE == kForward && k > 0) {
            store_tile(k - 1);
            __syncthreads();                               // its buffer may be written again
        }
        if (k + 1 < tiles) {
            load_tile(k + 1);
            load_bc(k + 1);
        }
        const int t0 = tile_at(k);
        T *raw = &sm.raw[k & 1][0][0];
        const float *Bs = sm.bc[k & 1][0], *Cs = sm.bc[k & 1][1];

        // what the recurrence needs of the lane's own token of group g: (Delta, Delta u), or
        // (Delta, dy) for the adjoint; returns u
        auto form = [&](int g) {
            const int r = g * LPC + q, t = t0 + r;
            float dt = 0.0f, x = 0.0f, u = 0.0f;
            if (t >= seq.start && t < seq.end && live) {
                u = to_f32(raw[r * CH + cl]);
                dt = softplus_acc(to_f32(raw[S::kRaw + r * CH + cl]) + bias);
                if (MODE == kAdjoint) {
                    x = u;
                    if (gz) {
                        const float z = to_f32(raw[2 * S::kRaw + r * CH + cl]);
                        x = u * (z * sigmoid(z));
                    }
                } else {
                    x = dt * u;
                }
            }
            *reinterpret_cast<float2 *>(&sm.ring[g & 1][cl * S::kRingRow + 2 * q]) = f2(dt, x);
            return u;
        };

        float u_next = form(MODE == kAdjoint ? GROUPS - 1 : 0);
#pragma unroll 1
        for (int gi = 0; gi < GROUPS; ++gi) {
            const int g = MODE == kAdjoint ? GROUPS - 1 - gi : gi;
            const float u_own = u_next;
            __syncwarp();
            const float4 *ring = reinterpret_cast<const float4 *>(&sm.ring[g & 1][cl * S::kRingRow]);
            float2 v[LPC];
#pragma unroll
            for (int i = 0; i < LPC / 2; ++i) {
                const float4 f = ring[i];
                v[2 * i] = f2(f.x, f.y);
                v[2 * i + 1] = f2(f.z, f.w);
            }
            if (gi + 1 < GROUPS) u_next = form(MODE == kAdjoint ? g - 1 : g + 1);

            float part[LPC];
            float Bq[LPC], Cq[LPC];
            if constexpr (NL == 1) {                       // the lane's state, all tokens of the group
                constexpr int W = LPC < 4 ? LPC : 4;
#pragma unroll
                for (int i = 0; i < LPC; i += W) {
#pragma unroll
                    for (int e = 0; e < W; ++e) {
                        if (HAS_B) Bq[i + e] = Bs[q * S::kBcRow + g * LPC + i + e];
                        if (HAS_C) Cq[i + e] = Cs[q * S::kBcRow + g * LPC + i + e];
                    }
                }
            }
#pragma unroll
            for (int ji = 0; ji < LPC; ++ji) {
                const int j = MODE == kAdjoint ? LPC - 1 - ji : ji;
                const int r = g * LPC + j, t = t0 + r;
                if (MODE != kAdjoint && p.ckpt && (j % kCkEvery) == 0 && (LPC >= kCkEvery || (r % kCkEvery) == 0) &&
                    t >= seq.start && t < seq.end && live) {
                    const int64_t row = b * ((p.seqs.L + kCkEvery - 1) / kCkEvery) + t / kCkEvery;
                    float *to = p.ckpt + (row * p.d + c) * N + q * NL;
#pragma unroll
                    for (int i = 0; i < NL; ++i) to[i] = h[i];
                }
                const float dt = v[j].x, x = v[j].y;
                if constexpr (NL == 1) {
                    const float a = ex2(dt * A2[0]);
                    if (MODE == kAdjoint) {
                        h[0] = a * fmaf(Cq[j], x, h[0]);
                    } else {
                        h[0] = fmaf(a, h[0], x * Bq[j]);
                        if (HAS_C) part[j] = h[0] * Cq[j];
                    }
                } else {
                    const float2 *B2 = reinterpret_cast<const float2 *>(Bs + r * N + q * NL);
                    const float2 *C2 = reinterpret_cast<const float2 *>(Cs + r * N + q * NL);
                    float2 acc = f2(0.0f, 0.0f);
#pragma unroll
                    for (int i = 0; i < NP; ++i) {
                        const float2 e = mul2(f2(A2[2 * i], A2[2 * i + 1]), f2(dt, dt));
                        const float2 a = f2(ex2(e.x), ex2(e.y));
                        float2 hh = f2(h[2 * i], h[2 * i + 1]);
                        if (MODE == kAdjoint) {
                            hh = mul2(a, fma2(C2[i], f2(x, x), hh));
                        } else {
                            hh = fma2(a, hh, mul2(B2[i], f2(x, x)));
                            if (HAS_C) acc = i == 0 ? mul2(C2[i], hh) : fma2(C2[i], hh, acc);
                        }
                        h[2 * i] = hh.x;
                        h[2 * i + 1] = hh.y;
                    }
                    part[j] = acc.x + acc.y;
                }
                if (MODE == kAdjoint && (t % kAdjEvery) == 0 && t > seq.start && t < seq.end && live) {
                    const int64_t row = b * ((p.seqs.L + kAdjEvery - 1) / kAdjEvery) + t / kAdjEvery - 1;
                    float *to = p.adj + (row * p.d + c) * N + q * NL;
#pragma unroll
                    for (int i = 0; i < NL; ++i) to[i] = h[i];
                }
            }
            if (MODE == kForward) {
                const float ch = reduce_scatter<LPC>(part, q);
                const int r = g * LPC + q;
                float y = fmaf(Dc, u_own, ch);
                if (gz) {
                    const float z = to_f32(raw[2 * S::kRaw + r * CH + cl]);
                    y *= z * sigmoid(z);
                }
                raw[r * CH + cl] = from_f32<T>(y);
            }
        }
        if (k + 1 < tiles) store_bc(k + 1);
    }
    if (MODE == kForward) {
        if (tiles > 0) {
            __syncthreads();
            store_tile(tiles - 1);
        }
    }
    if (MODE != kStates && p.state_out && live) {
        float *to = p.state_out + (seq.slot * p.d + c) * N + q * NL;
#pragma unroll
        for (int i = 0; i < NL; ++i) to[i] = h[i];
    }
}

}  // namespace

// Lanes a channel's states are spread over (N = 16: 4, 8 or 16, N = 8: 4 or 8), by the
// number of channels over all sequences.  Spreading wider costs issue slots (sums over
// more lanes, fewer packed pairs), spreading less leaves schedulers without a warp.
inline int causal_lanes(int N, int64_t channels) {
    if (N < 8) return N;
    if (channels >= 8 * 1184) return 4;
    if (N == 8 || channels >= 4 * 592) return 8;
    return 16;
}
template <int MODE>
vim_status launch_pass(const CausalArgs &a, int N, vim_dtype dt, cudaStream_t stream);

}  // namespace vimscan
