// Forward of the residual block's norms, bf16 tensors.
#include "moe_block_fwd.cuh"

namespace moe {
template cudaError_t launch_block_fwd_types<__nv_bfloat16, __nv_bfloat16>(BlockArgs, bool, int, cudaStream_t);
}  // namespace moe
