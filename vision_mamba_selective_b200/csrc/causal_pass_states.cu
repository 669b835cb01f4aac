// causal_pass_states.cu -- the causal scan's pass kernel, mode kStates.
#include "causal_pass.cuh"

namespace vimscan {
template vim_status launch_pass<kStates>(const CausalArgs &, int, vim_dtype, cudaStream_t);
}
