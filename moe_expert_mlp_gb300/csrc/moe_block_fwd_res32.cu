// Forward of the residual block's norms, bf16 tensors about an fp32 residual.
#include "moe_block_fwd.cuh"

namespace moe {
template cudaError_t launch_block_fwd_types<__nv_bfloat16, float>(BlockArgs, bool, int, cudaStream_t);
}  // namespace moe
