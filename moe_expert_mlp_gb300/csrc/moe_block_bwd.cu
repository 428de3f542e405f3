// Backward of the residual block's norms: the kernel over the rows
// (moe_block_bwd.cuh), then the sums over its blocks that give the parameters'
// gradients.
#include "moe_block.cuh"

namespace moe {
namespace {

// Adds the blocks' partials channel by channel, and turns the sums into the
// parameters' gradients.  32 channels a block; its 32 warps share the partials
// of each sum, and every thread has all of its own in flight at once.  Started
// while the rows' kernel still runs (programmatic launch) it waits for its end.
__global__ void __launch_bounds__(1024) k_block_bwd_finish(const __grid_constant__ BlockArgs p,
                                                           const __grid_constant__ BlockGrads o) {
  __shared__ float sums[4][32][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  wait_for_previous();
  constexpr int kEach = (kBlockBwdMaxParts + 31) / 32;
  for (int a = 0; a < o.acc; ++a) {
    float v[kEach], s = 0.0f;
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
      const int i = warp + 32 * j;
      v[j] = c < p.d && i < o.parts
                 ? p.part[(static_cast<long long>(i) * o.acc + a) * p.d + c] : 0.0f;
    }
#pragma unroll
    for (int j = 0; j < kEach; ++j) s += v[j];
    sums[a][warp][lane] = s;
  }
  __syncthreads();
  if (warp != 0 || c >= p.d) return;
  float S[4];
  for (int a = 0; a < o.acc; ++a) {
    S[a] = 0.0f;
    for (int i = 0; i < 32; ++i) S[a] += sums[a][i][lane];
  }
  auto param = [&](const void* w, float absent) {
    if (w == nullptr) return absent;
    return p.p32 ? static_cast<const float*>(w)[c]
                 : __bfloat162float(static_cast<const __nv_bfloat16*>(w)[c]);
  };
  auto put = [&](void* to, float v) {
    if (to == nullptr) return;
    if (p.p32)
      static_cast<float*>(to)[c] = v;
    else
      static_cast<__nv_bfloat16*>(to)[c] = __float2bfloat16_rn(v);
  };
  int a = 0;
  if (o.pre) {
    put(o.dpre_w, S[0]);
    if (o.bias) put(o.dpre_b, S[1]);
    a = o.bias ? 2 : 1;
  }
  if (o.post) {
    const float S1 = S[a], S0 = o.bias ? S[a + 1] : 0.0f;
    float scale = p.branch_scale;
    if (p.gate == MOE_GATE_CHANNEL) {
      const float gv = gate_act(p.gate_act, param(p.gate_rows.p, 1.0f));
      scale *= gv;
      const float w = p.post.w != nullptr ? param(p.post.w, 1.0f) + p.post.off : 1.0f;
      put(o.dgate, p.branch_scale * (w * S1 + param(p.post.b, 0.0f) * S0) *
                       gate_slope(p.gate_act, gv));
    }
    put(o.dpost_w, scale * S1);
    if (o.bias) put(o.dpost_b, scale * S0);
  }
}

}  // namespace

cudaError_t launch_block_bwd(const BlockArgs& a, BlockGrads o, int dtype, int res_dtype, int sms,
                             cudaStream_t s) {
  o.acc = (o.pre + o.post) * (o.bias ? 2 : 1);
  cudaError_t e;
  if (dtype == MOE_DTYPE_FP32)
    e = launch_block_bwd_types<float, float>(a, o, sms, s);
  else if (res_dtype == MOE_DTYPE_FP32)
    e = launch_block_bwd_types<__nv_bfloat16, float>(a, o, sms, s);
  else
    e = launch_block_bwd_types<__nv_bfloat16, __nv_bfloat16>(a, o, sms, s);
  const bool any = o.dpre_w || o.dpre_b || o.dpost_w || o.dpost_b || o.dgate;
  if (e == cudaSuccess && any) {
    e = launch_dependent(k_block_bwd_finish, (a.d + 31) / 32, 1024, s, a, o);
  }
  return e;
}

}  // namespace moe
