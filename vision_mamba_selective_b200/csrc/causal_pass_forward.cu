// causal_pass_forward.cu -- the causal scan's pass kernel, mode kForward.
#include "causal_pass.cuh"

namespace vimscan {
template vim_status launch_pass<kForward>(const CausalArgs &, int, vim_dtype, cudaStream_t);
}
