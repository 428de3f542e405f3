// Backward of the residual block's norms, fp32 tensors.
#include "moe_block_bwd.cuh"

namespace moe {
template cudaError_t launch_block_bwd_types<float, float>(BlockArgs, BlockGrads&, int, cudaStream_t);
}  // namespace moe
