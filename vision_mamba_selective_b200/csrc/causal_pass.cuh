// causal_pass.cuh -- instantiation and launch of causal_pass for one mode; included by one
// translation unit per mode, which compile in parallel.
#pragma once

#include "causal_kernels.cuh"

namespace vimscan {
namespace {

template <typename T, int N, int NL, int SEG, int MODE>
vim_status launch_pass_v(const CausalArgs &a, int warps, cudaStream_t stream) {
    using S = PassWarp<N, NL, SEG>;
    const int64_t grid = (int64_t)a.seqs.n * ((a.d + S::kCh - 1) / S::kCh);
    if (grid > INT32_MAX) return VIM_ERR_UNSUPPORTED;
    constexpr bool ALWAYS = MODE != kForward;              // the other modes are there to keep states
    auto kernel = ALWAYS || a.ckpt ? (a.vec_bc ? causal_pass<T, N, NL, SEG, MODE, true, true> : causal_pass<T, N, NL, SEG, MODE, true, false>)
                                   : (a.vec_bc ? causal_pass<T, N, NL, SEG, MODE, ALWAYS, true> : causal_pass<T, N, NL, SEG, MODE, ALWAYS, false>);
    static_assert(kPassWarps * sizeof(S) <= 48 * 1024, "no opt-in for shared memory");
    kernel<<<(unsigned)grid, 32 * warps, warps * sizeof(S), stream>>>(a);
    return cudaGetLastError() == cudaSuccess ? VIM_OK : VIM_ERR_CUDA;
}

template <typename T, int MODE>
vim_status launch_pass_t(const CausalArgs &a, int N, cudaStream_t stream) {
    const Seqs &q = a.seqs;
    const PassPlan pl = pass_plan(MODE, N, (int64_t)q.n * ((a.d + 7) / 8 * 8), q.cu != nullptr, q.cu ? q.L / q.n : q.L, q.L);
    switch (N) {
        case 2: return launch_pass_v<T, 2, 2, 8, MODE>(a, pl.warps, stream);
        case 4: return launch_pass_v<T, 4, 2, 8, MODE>(a, pl.warps, stream);
        case 8: return launch_pass_v<T, 8, 4, 8, MODE>(a, pl.warps, stream);
        default:
            if (pl.states == 8) return launch_pass_v<T, 16, 8, 4, MODE>(a, pl.warps, stream);
            if constexpr (MODE == kForward) {
                if (pl.states == 2) return launch_pass_v<T, 16, 2, kLongSeg, MODE>(a, pl.warps, stream);
                if (pl.seg == kLongSeg) return launch_pass_v<T, 16, 4, kLongSeg, MODE>(a, pl.warps, stream);
            }
            // (the adjoint, which has no other plan here, always in long segments)
            return launch_pass_v<T, 16, 4, MODE == kAdjoint ? kLongSeg : kSeg, MODE>(a, pl.warps, stream);
    }
}

}  // namespace

template <int MODE>
vim_status launch_pass(const CausalArgs &a, int N, vim_dtype dt, cudaStream_t stream) {
    return dt == VIM_F32 ? launch_pass_t<float, MODE>(a, N, stream) : launch_pass_t<__nv_bfloat16, MODE>(a, N, stream);
}

}  // namespace vimscan
