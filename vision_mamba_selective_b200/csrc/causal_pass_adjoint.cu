// causal_pass_adjoint.cu -- the causal scan's pass kernel, mode kAdjoint.
#include "causal_pass.cuh"

namespace vimscan {
template vim_status launch_pass<kAdjoint>(const CausalArgs &, int, vim_dtype, cudaStream_t);
}
