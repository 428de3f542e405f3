// Forward of the residual block's norms: the pre norm x = N1(r), and the post
// norm r' = a r + b G (*) N2(y) with the next block's norm x' = N1(r') in the
// same pass, y read as rows or combined from the routed expert rows.
//
// Bound by HBM: per channel a few operations against 4 to 16 bytes.  A row is
// read once into registers, its sums are taken there, and what follows from
// them is stored.
#include "moe_block.cuh"

namespace moe {
namespace {

// Statistics of the row held in v: mean (layer norm) and 1/sqrt(. + eps).
// The layer norm's variance sums squares about the mean, from registers.
template <int NV>
__device__ __forceinline__ void row_stats(const BlockArgs& p, const BlockNorm& n, Group& g,
                                          const UnitMap (&m)[NV], const float (&v)[NV][8],
                                          float& mu, float& rstd) {
  const float inv = 1.0f / static_cast<float>(p.d);
  mu = 0.0f;
  if (n.kind == MOE_NORM_LAYER) {
    float s[1] = {0.0f};
#pragma unroll
    for (int u = 0; u < NV; ++u)
#pragma unroll
      for (int e = 0; e < 8; ++e) s[0] += v[u][e];   // 0 past the row's end
    group_sum(g, s);
    mu = s[0] * inv;
  }
  float q[1] = {0.0f};
#pragma unroll
  for (int u = 0; u < NV; ++u)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float c = e < m[u].n ? v[u][e] - mu : 0.0f;
      q[0] += c * c;
    }
  group_sum(g, q);
  rstd = 1.0f / sqrtf(q[0] * inv + n.eps);
}

template <int NV>
__device__ __forceinline__ void normalize(const BlockArgs& p, const BlockNorm& n, Group& g,
                                          const UnitMap (&m)[NV], float (&v)[NV][8]) {
  float mu, rstd;
  row_stats<NV>(p, n, g, m, v, mu, rstd);
#pragma unroll
  for (int u = 0; u < NV; ++u) {
    float w[8], b[8];
    load_param(n.w, p, m[u], n.off, 1.0f, w);
    load_param(n.b, p, m[u], 0.0f, 0.0f, b);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[u][e] = (v[u][e] - mu) * rstd * w[e] + b[e];
  }
}

// y[t] from the expert rows, fp32 in slot order.
template <typename TA, int NV>
__device__ __forceinline__ void combine_rows(const BlockArgs& p, int t, const Group& g,
                                             const UnitMap (&m)[NV], float (&v)[NV][8]) {
#pragma unroll
  for (int u = 0; u < NV; ++u)
#pragma unroll
    for (int e = 0; e < 8; ++e) v[u][e] = 0.0f;
  const long long base = static_cast<long long>(t) * p.k;
#pragma unroll 4
  for (int s = 0; s < p.k; ++s) {
    const int r = __ldg(p.row_of + base + s);
    const float w = __ldg(p.topk_w + base + s);
    if (r < 0 || r >= p.capacity) {
      if (g.lane == 0) atomicOr(p.status, MOE_DEV_BAD_OFFSETS);
      continue;
    }
    const TA* row = row_ptr<TA>(p.y, r);
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      float q[8];
      load_unit(row, m[u], p.vec, q);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[u][e] += w * q[e];
    }
  }
}

template <typename TA, typename TR, int NV, bool POST>
__global__ void __launch_bounds__(kBlockThreads) k_block_fwd(const __grid_constant__ BlockArgs p) {
  __shared__ float4 red[2 * kBlockThreads / 32];
  Group g = make_group(p, red);
  const int groups = blockDim.x / p.tpr;
  UnitMap m[NV];
#pragma unroll
  for (int u = 0; u < NV; ++u) m[u] = unit_map(p, g.lane, u);
  for (int t = blockIdx.x * groups + g.id; t < p.T; t += gridDim.x * groups) {
    float v[NV][8];
    if constexpr (POST) {
      if (p.row_of != nullptr) {
        combine_rows<TA, NV>(p, t, g, m, v);
        if (p.y_out.p != nullptr) {
#pragma unroll
          for (int u = 0; u < NV; ++u) store_unit(row_ptr<TA>(p.y_out, t), m[u], p.vec, v[u]);
        }
      } else {
#pragma unroll
        for (int u = 0; u < NV; ++u) load_unit(row_ptr<const TA>(p.y, t), m[u], p.vec, v[u]);
      }
      float r[NV][8];
#pragma unroll
      for (int u = 0; u < NV; ++u) load_unit(row_ptr<const TR>(p.res, t), m[u], p.vec, r[u]);
      if (p.post.kind != MOE_NORM_NONE) normalize<NV>(p, p.post, g, m, v);
      float gt = 1.0f;
      if (p.gate == MOE_GATE_TOKEN)
        gt = gate_act(p.gate_act, *row_ptr<const float>(p.gate_rows, t));
#pragma unroll
      for (int u = 0; u < NV; ++u) {
        if (p.gate >= MOE_GATE_CHANNEL && p.gate != MOE_GATE_TOKEN) {
          float q[8];
          if (p.gate == MOE_GATE_CHANNEL)
            load_param(p.gate_rows.p, p, m[u], 0.0f, 1.0f, q);
          else
            load_unit(row_ptr<const TA>(p.gate_rows, t), m[u], p.vec, q);
#pragma unroll
          for (int e = 0; e < 8; ++e) v[u][e] *= gate_act(p.gate_act, q[e]);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e)
          v[u][e] = e < m[u].n ? p.res_scale * r[u][e] + p.branch_scale * gt * v[u][e] : 0.0f;
        store_unit(row_ptr<TR>(p.res_out, t), m[u], p.vec, v[u]);
      }
      if (p.x.p == nullptr) continue;
    } else {
#pragma unroll
      for (int u = 0; u < NV; ++u) load_unit(row_ptr<const TR>(p.res, t), m[u], p.vec, v[u]);
    }
    normalize<NV>(p, p.pre, g, m, v);
#pragma unroll
    for (int u = 0; u < NV; ++u) store_unit(row_ptr<TA>(p.x, t), m[u], p.vec, v[u]);
  }
}

template <typename TA, typename TR, int NV>
cudaError_t launch_nv(const BlockArgs& a, bool post, int threads, int blocks, cudaStream_t s) {
  if (post)
    k_block_fwd<TA, TR, NV, true><<<blocks, threads, 0, s>>>(a);
  else
    k_block_fwd<TA, TR, NV, false><<<blocks, threads, 0, s>>>(a);
  return cudaGetLastError();
}

template <typename TA, typename TR>
cudaError_t launch_types(const BlockArgs& a, bool post, cudaStream_t s) {
  const int groups = max(1, 256 / a.tpr);
  const int threads = groups * a.tpr, blocks = (a.T + groups - 1) / groups;
  if (a.nv == 1) return launch_nv<TA, TR, 1>(a, post, threads, blocks, s);
  if (a.nv == 2) return launch_nv<TA, TR, 2>(a, post, threads, blocks, s);
  return launch_nv<TA, TR, 4>(a, post, threads, blocks, s);
}

}  // namespace

cudaError_t launch_block_fwd(const BlockArgs& a, int dtype, int res_dtype, bool post,
                             cudaStream_t s) {
  if (dtype == MOE_DTYPE_FP32) return launch_types<float, float>(a, post, s);
  if (res_dtype == MOE_DTYPE_FP32) return launch_types<__nv_bfloat16, float>(a, post, s);
  return launch_types<__nv_bfloat16, __nv_bfloat16>(a, post, s);
}

}  // namespace moe
