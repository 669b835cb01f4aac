// causal.cu -- entry points of the causal selective scan (declared in include/vimscan.h)
// and its single-token kernel.
#include "causal_kernels.cuh"

#include <cstring>

namespace vimscan {
namespace {

// ----------------------------------------------------------------------------
// one token per sequence
// ----------------------------------------------------------------------------
// Bound by the state's traffic: 8 N bytes read and written per (sequence, channel) against
// 4 elements of activations.  A lane holds 4 states (one 16-byte load and store, whole
// lines per warp), N / 4 lanes a channel; Delta and the gate are formed by each of them,
// which costs nothing beside the loads.
struct StepArgs {
    vim_rows u, delta, z, B, C, y;
    const float *A, *D, *bias;
    Seqs seqs;
    const float *state;
    float *state_out;
    int d;
};
constexpr int kStepThreads = 128;

template <typename T, int N>
__global__ void __launch_bounds__(kStepThreads) causal_step(const StepArgs p) {
    constexpr int NL = N < 4 ? N : 4, LPC = N / NL, CH = kStepThreads / LPC;
    const int blocks = (p.d + CH - 1) / CH;
    const int64_t b = blockIdx.x / blocks;
    const int q = threadIdx.x % LPC, c = (int)(blockIdx.x % blocks) * CH + threadIdx.x / LPC;
    const Seq seq = sequence(p.seqs, (int)b);
    if (seq.slot < 0) return;
    const bool live = c < p.d;
    float part = 0.0f, u = 0.0f;
    if (live) {
        const int64_t at = (seq.slot * p.d + c) * N + q * NL;
        const float *hp = p.state + at, *Ap = p.A + (int64_t)c * N + q * NL;
        const T *Bp = static_cast<const T *>(p.B.data) + b * p.B.batch_stride + q * NL;
        const T *Cp = static_cast<const T *>(p.C.data) + b * p.C.batch_stride + q * NL;
        float h[NL], A[NL];
        if constexpr (NL == 4) {
            const float4 hv = *reinterpret_cast<const float4 *>(hp);
            const float4 av = *reinterpret_cast<const float4 *>(Ap);
            h[0] = hv.x, h[1] = hv.y, h[2] = hv.z, h[3] = hv.w;
            A[0] = av.x, A[1] = av.y, A[2] = av.z, A[3] = av.w;
        } else {
#pragma unroll
            for (int i = 0; i < NL; ++i) h[i] = hp[i], A[i] = Ap[i];
        }
        if (seq.fresh) {
#pragma unroll
            for (int i = 0; i < NL; ++i) h[i] = 0.0f;
        }
        u = to_f32(static_cast<const T *>(p.u.data)[b * p.u.batch_stride + c]);
        const float dt = softplus_acc(to_f32(static_cast<const T *>(p.delta.data)[b * p.delta.batch_stride + c]) +
                                      p.bias[c]);
        const float du = dt * u;
#pragma unroll
        for (int i = 0; i < NL; ++i) {
            h[i] = fmaf(decay(A[i] * kLog2e, dt), h[i], du * to_f32(Bp[i]));
            part = fmaf(to_f32(Cp[i]), h[i], part);
        }
        float *ho = p.state_out + at;
        if constexpr (NL == 4) {
            *reinterpret_cast<float4 *>(ho) = make_float4(h[0], h[1], h[2], h[3]);
        } else {
#pragma unroll
            for (int i = 0; i < NL; ++i) ho[i] = h[i];
        }
    }
#pragma unroll
    for (int o = 1; o < LPC; o <<= 1) part += __shfl_xor_sync(0xffffffffu, part, o);
    if (live && q == 0) {
        float y = fmaf(p.D[c], u, part);
        if (p.z.data) {
            const float z = to_f32(static_cast<const T *>(p.z.data)[b * p.z.batch_stride + c]);
            y *= z * sigmoid(z);
        }
        static_cast<T *>(const_cast<void *>(p.y.data))[b * p.y.batch_stride + c] = from_f32<T>(y);
    }
}

vim_status check_scan(const vim_rows &u, const vim_rows &delta, const vim_rows &z, const vim_rows &B,
                      const vim_rows &C, const float *A, const float *D, const float *bias, vim_dtype dt) {
    if (bad_rows(u, dt) || bad_rows(delta, dt) || bad_rows(B, dt) || bad_rows(C, dt) || (z.data && bad_rows(z, dt)))
        return VIM_ERR_INVALID_ARG;
    if (!A || !D || !bias || misaligned(A, 16) || misaligned(D, 4) || misaligned(bias, 4)) return VIM_ERR_INVALID_ARG;
    return VIM_OK;
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
    st = make_seqs(seqs, batch, L, 16, &a.seqs);
    if (st != VIM_OK) return st;
    if (a.seqs.n == 0 || d_inner == 0) return VIM_OK;
    if (L > 0) {
        st = check_scan(u, delta, z, B, C, A, D, delta_bias, dt);
        if (st != VIM_OK) return st;
        if (bad_out(y, dt, batch, L, d_inner) || misaligned(ckpt, 16)) return VIM_ERR_INVALID_ARG;
    } else if (!A || !delta_bias || !D) {
        return VIM_ERR_INVALID_ARG;
    }
    a.u = u, a.delta = delta, a.z = z, a.B = B, a.C = C, a.y = y;
    a.A = A, a.D = D, a.bias = delta_bias;
    a.state = static_cast<const float *>(seqs ? seqs->state : nullptr);
    a.state_out = static_cast<float *>(seqs ? seqs->state_out : nullptr);
    a.ckpt = ckpt;
    a.d = d_inner;
    a.vec_bc = lane_vectors(B, dt, batch, L, d_state) && lane_vectors(C, dt, batch, L, d_state);
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
    st = make_seqs(&rows, batch, 1, 16, &a.seqs);
    if (st != VIM_OK) return st;
    if (batch == 0 || d_inner == 0) return VIM_OK;
    if (!rows.state) return VIM_ERR_INVALID_ARG;
    st = check_scan(u, delta, z, B, C, A, D, delta_bias, dt);
    if (st != VIM_OK) return st;
    if (bad_out(y, dt, batch, 1, d_inner)) return VIM_ERR_INVALID_ARG;
    a.u = u, a.delta = delta, a.z = z, a.B = B, a.C = C, a.y = y;
    a.A = A, a.D = D, a.bias = delta_bias;
    a.state = static_cast<const float *>(rows.state);
    a.state_out = static_cast<float *>(rows.state_out);
    a.d = d_inner;
    auto launch = [&](auto kernel, int per) {
        const int64_t grid = (int64_t)batch * ((d_inner + per - 1) / per);
        if (grid > INT32_MAX) return VIM_ERR_UNSUPPORTED;
        kernel<<<(unsigned)grid, kStepThreads, 0, stream>>>(a);
        return cudaGetLastError() == cudaSuccess ? VIM_OK : VIM_ERR_CUDA;
    };
    const bool f = dt == VIM_F32;
    switch (d_state) {
        case 2: return f ? launch(causal_step<float, 2>, 128) : launch(causal_step<__nv_bfloat16, 2>, 128);
        case 4: return f ? launch(causal_step<float, 4>, 128) : launch(causal_step<__nv_bfloat16, 4>, 128);
        case 8: return f ? launch(causal_step<float, 8>, 64) : launch(causal_step<__nv_bfloat16, 8>, 64);
        default: return f ? launch(causal_step<float, 16>, 32) : launch(causal_step<__nv_bfloat16, 16>, 32);
    }
}

}  // extern "C"
