// Forward of the residual block's norms, fp32 tensors.
#include "moe_block_fwd.cuh"

namespace moe {
template cudaError_t launch_block_fwd_types<float, float>(BlockArgs, bool, int, cudaStream_t);
}  // namespace moe
