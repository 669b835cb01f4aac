// causal_pass.cuh -- instantiation and launch of causal_pass for one mode; included by one
// translation unit per mode, which compile in parallel.
#pragma once

#include "causal_kernels.cuh"

namespace vimscan {
namespace {

template <typename T, int N, int NL, int MODE>
vim_status launch_pass_v(const CausalArgs &a, cudaStream_t stream) {
    constexpr int TOK = 32;
    using S = PassStage<T, N, NL, TOK>;
    const int64_t grid = (int64_t)a.seqs.n * ((a.d + S::kCh - 1) / S::kCh);
    if (grid > INT32_MAX) return VIM_ERR_UNSUPPORTED;
    auto kernel = causal_pass<T, N, NL, TOK, MODE>;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(S)) != cudaSuccess)
        return VIM_ERR_CUDA;
    kernel<<<(unsigned)grid, kPassThreads, sizeof(S), stream>>>(a);
    return cudaGetLastError() == cudaSuccess ? VIM_OK : VIM_ERR_CUDA;
}

template <typename T, int MODE>
vim_status launch_pass_t(const CausalArgs &a, int N, cudaStream_t stream) {
    const int lanes = causal_lanes(N, (int64_t)a.seqs.n * a.d);
    switch (N) {
        case 2: return launch_pass_v<T, 2, 1, MODE>(a, stream);
        case 4: return launch_pass_v<T, 4, 1, MODE>(a, stream);
        case 8: return lanes == 4 ? launch_pass_v<T, 8, 2, MODE>(a, stream) : launch_pass_v<T, 8, 1, MODE>(a, stream);
        default:
            return lanes == 4   ? launch_pass_v<T, 16, 4, MODE>(a, stream)
                   : lanes == 8 ? launch_pass_v<T, 16, 2, MODE>(a, stream)
                                : launch_pass_v<T, 16, 1, MODE>(a, stream);
    }
}

}  // namespace

template <int MODE>
vim_status launch_pass(const CausalArgs &a, int N, vim_dtype dt, cudaStream_t stream) {
    return dt == VIM_F32 ? launch_pass_t<float, MODE>(a, N, stream) : launch_pass_t<__nv_bfloat16, MODE>(a, N, stream);
}

}  // namespace vimscan
