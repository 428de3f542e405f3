// Backward of the residual block's norms, bf16 tensors about an fp32 residual.
#include "moe_block_bwd.cuh"

namespace moe {
template cudaError_t launch_block_bwd_types<__nv_bfloat16, float>(BlockArgs, BlockGrads&, int, cudaStream_t);
}  // namespace moe
