// causal.cu -- entry points of the causal selective scan (declared in include/vimscan_causal.h)
// and its single-token kernel.
#include "causal_kernels.cuh"

#include <algorithm>
#include <cstring>

namespace vimscan {
namespace {

// ----------------------------------------------------------------------------
// one token per sequence
// ----------------------------------------------------------------------------
// Bound by the state's traffic: 8 N bytes read and written per (sequence, channel) against
// 4 elements of activations.  A lane holds 4 states (one 16-byte load and store, whole
// lines per warp), LPC = N / 4 lanes a channel.  A warp takes its channels through up to
// 32 sequences, LPC at a time: A is read once, the slots of all of them with one load, and
// the states and inputs of the next ones are on their way while the present ones are
// computed (without that the chain slot -> state -> store leaves memory idle half of the
// time).  Each of a channel's lanes forms Delta and the gate of one of the LPC sequences,
// exchanged by shuffles, so that no lane repeats another's work.  256 x 4096, N = 16, bf16:
// 28 us on the device, 22 at the copy rate for the 143 MB.
struct StepArgs {
    vim_rows u, delta, z, B, C, y;         // row b: sequence b
    const float *A, *D, *bias;
    Seqs seqs;
    const float *state;
    float *state_out;
    int d, per_warp;                       // sequences a warp takes: a multiple of LPC, at most 32
};
constexpr int kStepWarps = 4;

template <typename T, int N, bool VEC>
__global__ void __launch_bounds__(32 * kStepWarps) causal_step(const StepArgs p) {
    constexpr int NL = N < 4 ? N : 4, LPC = N / NL, CH = 32 / LPC, R = LPC;
    constexpr int WB = NL * (int)sizeof(T) / 4;            // words of a lane's B (C)
    const int w = threadIdx.x / 32, lane = threadIdx.x % 32, q = lane % LPC;
    const int blocks = (p.d + CH * kStepWarps - 1) / (CH * kStepWarps);
    const int c_warp = ((int)(blockIdx.x % blocks) * kStepWarps + w) * CH, c_at = c_warp + lane / LPC;
    if (c_warp >= p.d) return;                             // (it would read what another warp writes in place)
    const int b0 = (int)(blockIdx.x / blocks) * p.per_warp, b1 = min(b0 + p.per_warp, p.seqs.n);
    const bool live = c_at < p.d;
    const int c = live ? c_at : p.d - 1;                   // channels past d repeat the last and write nothing

    int slot_of = -1;                                      // of sequence b0 + lane; -1 none, -2 - slot: fresh
    if (b0 + lane < b1) {
        const Seq seq = sequence(p.seqs, b0 + lane);
        slot_of = seq.slot < 0 ? -1 : seq.fresh ? -2 - (int)seq.slot : (int)seq.slot;
    }
    const RowsOf<T, kInPlaceFree> gu(p.u, 0, c), gd(p.delta, 0, c), gz(p.z.data ? p.z : p.u, 0, c);   // y may lie over them
    const RowsOf<T> gy(p.y, 0, c), gB(p.B, 0, q * NL), gC(p.C, 0, q * NL);
    const float bias = p.bias[c], Dc = p.D[c];
    float A[NL];
#pragma unroll
    for (int i = 0; i < NL; ++i) A[i] = decay_rate(p.A[(int64_t)c * N + q * NL + i]);
    const int mine = c * N + q * NL, row = p.d * N;        // the lane's states in a slot's row

    float h[R][NL];
    uint32_t wb[R][WB], wc[R][WB], ru = 0, rd = 0, rz = 0;
    auto fetch = [&](int b) {                              // sequences b .. b + R - 1; those past b1 read the last
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int slot = __shfl_sync(0xffffffffu, slot_of, min(b + r, b1 - 1) - b0), br = min(b + r, b1 - 1);
            const float *from = p.state + (int64_t)max(slot, 0) * row + mine;
#pragma unroll
            for (int i = 0; i < NL; ++i) h[r][i] = 0.0f;
            if (slot >= 0) {
                if constexpr (NL == 4) {
                    const float4 v = *reinterpret_cast<const float4 *>(from);
                    h[r][0] = v.x, h[r][1] = v.y, h[r][2] = v.z, h[r][3] = v.w;
                } else {
#pragma unroll
                    for (int i = 0; i < NL; ++i) h[r][i] = from[i];
                }
            }
            if constexpr (VEC) gB.template words<WB>(br, wb[r]), gC.template words<WB>(br, wc[r]);
            else gB.template gather<WB>(br, wb[r]), gC.template gather<WB>(br, wc[r]);
        }
        const int own = min(b + q, b1 - 1);
        ru = gu.raw(own), rd = gd.raw(own), rz = gz.raw(own);
    };
    fetch(b0);
#pragma unroll 1
    for (int b = b0; b < b1; b += R) {
        float g[R][NL], Bv[R][NL], Cv[R][NL];
#pragma unroll
        for (int r = 0; r < R; ++r) {
#pragma unroll
            for (int i = 0; i < NL; ++i) {
                g[r][i] = h[r][i];
                Bv[r][i] = word_f32<T>(wb[r][i * (int)sizeof(T) / 4], i);
                Cv[r][i] = word_f32<T>(wc[r][i * (int)sizeof(T) / 4], i);
            }
        }
        const float u = bits_f32<T>(ru), dt = softplus_acc(bits_f32<T>(rd) + bias), z = bits_f32<T>(rz), du = dt * u;
        if (b + R < b1) fetch(b + R);
        float part[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const float dr = __shfl_sync(0xffffffffu, dt, lane - q + r), xr = __shfl_sync(0xffffffffu, du, lane - q + r);
            part[r] = 0.0f;
#pragma unroll
            for (int i = 0; i < NL; ++i) {
                g[r][i] = fmaf(decay(A[i], dr), g[r][i], xr * Bv[r][i]);
                part[r] = fmaf(Cv[r][i], g[r][i], part[r]);
            }
            const int code = __shfl_sync(0xffffffffu, slot_of, min(b + r, b1 - 1) - b0);
            if (live && b + r < b1 && code != -1) {
                float *to = p.state_out + (int64_t)(code < 0 ? -2 - code : code) * row + mine;
                if constexpr (NL == 4) {
                    *reinterpret_cast<float4 *>(to) = make_float4(g[r][0], g[r][1], g[r][2], g[r][3]);
                } else {
#pragma unroll
                    for (int i = 0; i < NL; ++i) to[i] = g[r][i];
                }
            }
        }
        float y = fmaf(Dc, u, reduce_scatter<R, 1>(part, q));
        if (p.z.data) y *= z * sigmoid(z);
        const int code = __shfl_sync(0xffffffffu, slot_of, min(b + q, b1 - 1) - b0);
        if (live && b + q < b1 && code != -1) gy.put(b + q, y);
    }
}

// the tensors of a call; y may be u, delta or z itself
bool bad_tensors(const vim_rows &u, const vim_rows &delta, const vim_rows &z, const vim_rows &B, const vim_rows &C,
                 const vim_rows &y, vim_dtype dt, int batch, int L, int d, int N) {
    if (bad_rows(u, dt) || bad_rows(delta, dt) || bad_rows(B, dt) || bad_rows(C, dt) || (z.data && bad_rows(z, dt)) ||
        bad_out(y, dt, batch, L, d))
        return true;
    return rows_clash(y, u, d, dt, batch, L) || rows_clash(y, delta, d, dt, batch, L) || rows_clash(y, z, d, dt, batch, L) ||
           rows_meet(y, d, B, N, dt, batch, L) || rows_meet(y, d, C, N, dt, batch, L);
}

}  // namespace
}  // namespace vimscan

using namespace vimscan;

extern "C" {

size_t causal_ckpt_bytes(int batch, int L, int d_inner, int d_state) {
    if (batch <= 0 || L <= 0 || d_inner <= 0 || !supported_state(d_state)) return 0;
    return (size_t)batch * ((L + kCkEvery - 1) / kCkEvery) * d_inner * d_state * sizeof(float);
}

vim_status causal_scan(const vim_scan_io *io, const float *A, const float *D, const float *delta_bias, int batch,
                       int L, int d_inner, int d_state, vim_dtype dt, const vim_sequences *seqs, float *ckpt,
                       cudaStream_t stream) {
    if (!io) return VIM_ERR_INVALID_ARG;
    const vim_rows &u = io->u, &delta = io->delta, &z = io->z, &B = io->B, &C = io->C, &y = io->y;
    vim_status st = check_sizes(batch, L, d_inner, dt);
    if (st != VIM_OK) return st;
    if (!supported_state(d_state)) return VIM_ERR_UNSUPPORTED;
    CausalArgs a;
    std::memset(&a, 0, sizeof(a));
    st = make_seqs(seqs, batch, L, 16, (int64_t)d_inner * d_state * sizeof(float), &a.seqs);
    if (st != VIM_OK) return st;
    if (ckpt && seqs && seqs->state) return VIM_ERR_INVALID_ARG;   // the derivative starts every sequence from zeros
    if (a.seqs.n == 0 || d_inner == 0) return VIM_OK;
    if (bad_params(A, D, delta_bias)) return VIM_ERR_INVALID_ARG;   // without tokens too: the kernel loads them first
    if (L > 0 && (bad_tensors(u, delta, z, B, C, y, dt, batch, L, d_inner, d_state) || misaligned(ckpt, 16)))
        return VIM_ERR_INVALID_ARG;
    a.u = u, a.delta = delta, a.z = z, a.B = B, a.C = C, a.y = y;
    a.A = A, a.D = D, a.bias = delta_bias;
    a.state = static_cast<const float *>(seqs ? seqs->state : nullptr);
    a.state_out = static_cast<float *>(seqs ? seqs->state_out : nullptr);
    a.ckpt = ckpt;
    a.d = d_inner;
    a.vec_bc = row_vectors(B, dt, batch, L, lane_states(d_state)) && row_vectors(C, dt, batch, L, lane_states(d_state));
    return launch_pass<kForward>(a, d_state, dt, stream);
}

vim_status causal_scan_step(const vim_scan_io *io, const float *A, const float *D, const float *delta_bias,
                            int batch, int d_inner, int d_state, vim_dtype dt, const vim_sequences *seqs,
                            cudaStream_t stream) {
    if (!io) return VIM_ERR_INVALID_ARG;
    const vim_rows &u = io->u, &delta = io->delta, &z = io->z, &B = io->B, &C = io->C, &y = io->y;
    vim_status st = check_sizes(batch, 1, d_inner, dt);
    if (st != VIM_OK) return st;
    if (!supported_state(d_state)) return VIM_ERR_UNSUPPORTED;
    if (!seqs) return VIM_ERR_INVALID_ARG;
    vim_sequences rows = *seqs;
    rows.cu_seqlens = nullptr;
    if (!rows.state_out) rows.state_out = const_cast<void *>(rows.state);
    StepArgs a;
    std::memset(&a, 0, sizeof(a));
    st = make_seqs(&rows, batch, 1, 16, (int64_t)d_inner * d_state * sizeof(float), &a.seqs);
    if (st != VIM_OK) return st;
    if (batch == 0 || d_inner == 0) return VIM_OK;
    if (!rows.state) return VIM_ERR_INVALID_ARG;
    if (bad_params(A, D, delta_bias) || bad_tensors(u, delta, z, B, C, y, dt, batch, 1, d_inner, d_state))
        return VIM_ERR_INVALID_ARG;
    // the kernel's rows are the sequences
    vim_rows in[6] = {u, delta, z, B, C, y};
    for (vim_rows &r : in) {
        r.row_stride = r.batch_stride;
        r.batch_stride = 0;
        if (r.row_stride > INT32_MAX / 4) return VIM_ERR_UNSUPPORTED;
    }
    if ((int64_t)d_inner * d_state > INT32_MAX) return VIM_ERR_UNSUPPORTED;
    a.u = in[0], a.delta = in[1], a.z = in[2], a.B = in[3], a.C = in[4], a.y = in[5];
    a.A = A, a.D = D, a.bias = delta_bias;
    a.state = static_cast<const float *>(rows.state);
    a.state_out = static_cast<float *>(rows.state_out);
    a.d = d_inner;
    // a warp's sequences: as many as leave about 12 warps an SM, in whole groups of its lanes
    const int lanes = d_state < 8 ? 1 : d_state / 4, per = 32 / lanes * kStepWarps;
    const int64_t blocks = (d_inner + per - 1) / per;
    const int64_t want = (int64_t)batch * blocks * kStepWarps / (148 * 12);
    a.per_warp = (int)std::max<int64_t>(lanes, std::min<int64_t>(32, want / lanes * lanes));
    const int64_t grid = ((int64_t)batch + a.per_warp - 1) / a.per_warp * blocks;
    if (grid > INT32_MAX) return VIM_ERR_UNSUPPORTED;
    auto launch = [&](auto kernel) {
        kernel<<<(unsigned)grid, 32 * kStepWarps, 0, stream>>>(a);
        return cudaGetLastError() == cudaSuccess ? VIM_OK : VIM_ERR_CUDA;
    };
    const int n = d_state < 4 ? d_state : 4;
    const bool vec = row_vectors(a.B, dt, 1, batch, n) && row_vectors(a.C, dt, 1, batch, n);
    auto launch_n = [&](auto f32_vec, auto f32_any, auto bf16_vec, auto bf16_any) {
        return dt == VIM_F32 ? (vec ? launch(f32_vec) : launch(f32_any)) : (vec ? launch(bf16_vec) : launch(bf16_any));
    };
    using bf16 = __nv_bfloat16;
    switch (d_state) {
        case 2: return launch_n(causal_step<float, 2, true>, causal_step<float, 2, false>, causal_step<bf16, 2, true>, causal_step<bf16, 2, false>);
        case 4: return launch_n(causal_step<float, 4, true>, causal_step<float, 4, false>, causal_step<bf16, 4, true>, causal_step<bf16, 4, false>);
        case 8: return launch_n(causal_step<float, 8, true>, causal_step<float, 8, false>, causal_step<bf16, 8, true>, causal_step<bf16, 8, false>);
        default: return launch_n(causal_step<float, 16, true>, causal_step<float, 16, false>, causal_step<bf16, 16, true>, causal_step<bf16, 16, false>);
    }
}

}  // extern "C"
