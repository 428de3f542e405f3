// Forward kernel of the residual block's norms: the pre norm x = N1(r), and
// the post norm r' = a r + b G (*) N2(y) with the next block's norm
// x' = N1(r') in the same pass, y read as rows or combined from the routed
// expert rows.  Instantiated type by type in moe_block_fwd_*.cu.
//
// Bound by HBM: a few operations a channel against 4 to 16 bytes.  A row is
// read once into registers, its sums are taken there, and what follows from
// them is stored.  Groups are small (about 128 threads with up to 8 units
// each) and blocks hold one row of a group at a time, so that several
// independent blocks share an SM: while one waits at its sums others have
// their loads in flight.  Parameters stay in L1, which the rows bypass.
//
// With few rows (HOIST) nothing hides the latency of one row, so the group is
// as large as the row allows and the parameters are fetched together with the
// row instead of after its sums.
#pragma once

#include "moe_block.cuh"

namespace moe {
namespace {

// Statistics of the row held in v: mean (layer norm) and 1/sqrt(. + eps).
// The layer norm's variance sums squares about the mean, from registers.
template <int NV, bool VEC>
__device__ __forceinline__ void row_stats(const BlockArgs& p, const BlockNorm& n, Group& g,
                                          const Unit<VEC> (&m)[NV], const float (&v)[NV][8],
                                          float& mu, float& rstd) {
  const float inv = 1.0f / static_cast<float>(p.d);
  float q[1] = {0.0f};
  mu = 0.0f;
  if (n.kind == MOE_NORM_LAYER) {
    float s[1] = {0.0f};
#pragma unroll
    for (int u = 0; u < NV; ++u)
#pragma unroll
      for (int e = 0; e < 8; ++e) s[0] += v[u][e];   // 0 past the row's end
    group_sum(g, s);
    mu = s[0] * inv;
#pragma unroll
    for (int u = 0; u < NV; ++u)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float c = m[u].has(e) ? v[u][e] - mu : 0.0f;
        q[0] += c * c;
      }
  } else {
#pragma unroll
    for (int u = 0; u < NV; ++u)
#pragma unroll
      for (int e = 0; e < 8; ++e) q[0] += v[u][e] * v[u][e];
  }
  group_sum(g, q);
  rstd = 1.0f / sqrtf(q[0] * inv + n.eps);
}

// Weight, bias and channel gate of a thread's units: fetched ahead (HOIST),
// or from L1 where they are used.
template <int NV, bool VEC, bool HOIST>
struct Params {
  float held[HOIST ? NV : 1][8];
  __device__ __forceinline__ void fetch(const void* w, const BlockArgs& p,
                                        const Unit<VEC> (&m)[NV], float off) {
    if constexpr (HOIST) {
#pragma unroll
      for (int u = 0; u < NV; ++u) load_param(w, p, m[u], off, 1.0f, held[u]);
    }
  }
  __device__ __forceinline__ void get(const void* w, const BlockArgs& p, const Unit<VEC>& m, int u,
                                      float off, float (&v)[8]) const {
    if constexpr (HOIST) {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = held[u][e];
    } else {
      load_param(w, p, m, off, 1.0f, v);
    }
  }
};

// v = xhat * (off + w) + b
template <int NV, bool VEC, bool HOIST>
__device__ __forceinline__ void normalize(const BlockArgs& p, const BlockNorm& n, Group& g,
                                          const Unit<VEC> (&m)[NV],
                                          const Params<NV, VEC, HOIST>& pw,
                                          const Params<NV, VEC, HOIST>& pb, float (&v)[NV][8]) {
  float mu, rstd;
  row_stats(p, n, g, m, v, mu, rstd);
#pragma unroll
  for (int u = 0; u < NV; ++u) {
    float w[8];
    pw.get(n.w, p, m[u], u, n.off, w);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[u][e] = (v[u][e] - mu) * rstd * w[e];
    if (n.b != nullptr) {
      float b[8];
      pb.get(n.b, p, m[u], u, 0.0f, b);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[u][e] += b[e];
    }
  }
}

// y[t] from the expert rows, fp32 in slot order; four rows' loads in flight.
template <typename TA, int NV, bool VEC>
__device__ __forceinline__ void combine_rows(const BlockArgs& p, int t, const Group& g,
                                             const Unit<VEC> (&m)[NV], float (&v)[NV][8]) {
#pragma unroll
  for (int u = 0; u < NV; ++u)
#pragma unroll
    for (int e = 0; e < 8; ++e) v[u][e] = 0.0f;
  const long long base = static_cast<long long>(t) * p.k;
  for (int s = 0; s < p.k; s += 4) {
    const TA* row[4];
    float w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      row[i] = nullptr;
      w[i] = 0.0f;
      if (s + i < p.k) {
        const int r = __ldg(p.row_of + base + s + i);
        w[i] = __ldg(p.topk_w + base + s + i);
        if (r >= 0 && r < p.capacity)
          row[i] = row_ptr<const TA>(p.y, r);
        else if (g.lane == 0)
          atomicOr(p.status, MOE_DEV_BAD_OFFSETS);
      }
    }
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      Raw<TA, VEC> q[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (row[i] != nullptr) q[i].template load<true>(row[i], m[u]);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (row[i] != nullptr) {
#pragma unroll
          for (int e = 0; e < 8; ++e) v[u][e] += w[i] * q[i].get(e);
        }
    }
  }
}

enum FwdMode { kPre, kPost, kRouted };

template <typename TA, typename TR, int NV, bool VEC, int MODE, bool HOIST>
__global__ void __launch_bounds__(HOIST ? kBlockThreads : kBlockThreads / 2)
    k_block_fwd(const __grid_constant__ BlockArgs p) {
  __shared__ float4 red[2 * kBlockThreads / 32];
  Group g = make_group(p, red);
  const int t = blockIdx.x * (blockDim.x / p.tpr) + g.id;
  if (t >= p.T) return;
  Unit<VEC> m[NV];
#pragma unroll
  for (int u = 0; u < NV; ++u) m[u] = Unit<VEC>(p, g.lane, u);
  Params<NV, VEC, HOIST> w1, b1, w2, b2, gc;
  float v[NV][8];
  if constexpr (MODE != kPre) {
    if constexpr (MODE == kPost) {
#pragma unroll
      for (int u = 0; u < NV; ++u) load_row(row_ptr<const TA>(p.y, t), m[u], v[u]);
    }
    Raw<TR, VEC> r[NV];
#pragma unroll
    for (int u = 0; u < NV; ++u) r[u].template load<true>(row_ptr<const TR>(p.res, t), m[u]);
    float gt = 1.0f;
    if (p.gate == MOE_GATE_TOKEN)
      gt = gate_act(p.gate_act, *row_ptr<const float>(p.gate_rows, t));
    gt *= p.branch_scale;
    w2.fetch(p.post.w, p, m, p.post.off);
    b2.fetch(p.post.b, p, m, 0.0f);
    if (p.gate == MOE_GATE_CHANNEL) gc.fetch(p.gate_rows.p, p, m, 0.0f);
    if (p.x.p != nullptr) {
      w1.fetch(p.pre.w, p, m, p.pre.off);
      b1.fetch(p.pre.b, p, m, 0.0f);
    }
    if constexpr (MODE == kRouted) {
      combine_rows<TA>(p, t, g, m, v);
      if (p.y_out.p != nullptr) {
#pragma unroll
        for (int u = 0; u < NV; ++u) store_unit(row_ptr<TA>(p.y_out, t), m[u], v[u]);
      }
    }
    if (p.post.kind != MOE_NORM_NONE) normalize(p, p.post, g, m, w2, b2, v);
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      if (p.gate == MOE_GATE_CHANNEL || p.gate == MOE_GATE_FULL) {
        float q[8];
        if (p.gate == MOE_GATE_CHANNEL)
          gc.get(p.gate_rows.p, p, m[u], u, 0.0f, q);
        else
          load_row(row_ptr<const TA>(p.gate_rows, t), m[u], q);
        if (p.gate_act != MOE_GATE_ACT_NONE) {
#pragma unroll
          for (int e = 0; e < 8; ++e) q[e] = gate_act(p.gate_act, q[e]);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) v[u][e] *= q[e];
      }
#pragma unroll
      for (int e = 0; e < 8; ++e)
        v[u][e] = m[u].has(e) ? p.res_scale * r[u].get(e) + gt * v[u][e] : 0.0f;
      store_unit(row_ptr<TR>(p.res_out, t), m[u], v[u]);
    }
    if (p.x.p == nullptr) return;
  } else {
#pragma unroll
    for (int u = 0; u < NV; ++u) load_row(row_ptr<const TR>(p.res, t), m[u], v[u]);
    w1.fetch(p.pre.w, p, m, p.pre.off);
    b1.fetch(p.pre.b, p, m, 0.0f);
  }
  normalize(p, p.pre, g, m, w1, b1, v);
#pragma unroll
  for (int u = 0; u < NV; ++u) store_unit(row_ptr<TA>(p.x, t), m[u], v[u]);
}

template <typename TA, typename TR, int NV, bool VEC, bool HOIST>
cudaError_t launch_nv(const BlockArgs& a, bool post, cudaStream_t s) {
  const int groups = max(1, 128 / a.tpr);
  const int threads = groups * a.tpr, blocks = (a.T + groups - 1) / groups;
  if (!post)
    k_block_fwd<TA, TR, NV, VEC, kPre, HOIST><<<blocks, threads, 0, s>>>(a);
  else if (a.row_of == nullptr)
    k_block_fwd<TA, TR, NV, VEC, kPost, HOIST><<<blocks, threads, 0, s>>>(a);
  else
    k_block_fwd<TA, TR, NV, VEC, kRouted, HOIST><<<blocks, threads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

template <typename TA, typename TR>
cudaError_t launch_block_fwd_types(BlockArgs a, bool post, int sms, cudaStream_t s) {
  const int units = (a.d + kUnit - 1) / kUnit;
  auto threads = [&](int nv) { return ((units + nv - 1) / nv + 31) / 32 * 32; };
  if (!a.vec) {
    const bool wide = units > 2 * kBlockThreads / 2;
    a.tpr = threads(wide ? 8 : 2);
    return wide ? launch_nv<TA, TR, 8, false, false>(a, post, s)
                : launch_nv<TA, TR, 2, false, false>(a, post, s);
  }
  if (a.T <= kFewRows * sms && units <= 2 * kBlockThreads) {
    const bool one = units <= kBlockThreads;
    a.tpr = threads(one ? 1 : 2);
    return one ? launch_nv<TA, TR, 1, true, true>(a, post, s)
               : launch_nv<TA, TR, 2, true, true>(a, post, s);
  }
  // units a thread: the count (of 1, 2, 3, 4, 7, 8) that leaves the fewest of
  // the group's places empty with at most 160 threads
  int nv = 8;
  float best = 0.0f;
  for (int n : {1, 2, 3, 4, 7, 8}) {
    const int tpr = threads(n);
    const float used = static_cast<float>(units) / (n * tpr);
    if (tpr <= 160 && used > best + 0.02f) best = used, nv = n;
  }
  a.tpr = threads(nv);
  switch (nv) {
    case 1: return launch_nv<TA, TR, 1, true, false>(a, post, s);
    case 2: return launch_nv<TA, TR, 2, true, false>(a, post, s);
    case 3: return launch_nv<TA, TR, 3, true, false>(a, post, s);
    case 4: return launch_nv<TA, TR, 4, true, false>(a, post, s);
    case 7: return launch_nv<TA, TR, 7, true, false>(a, post, s);
    default: return launch_nv<TA, TR, 8, true, false>(a, post, s);
  }
}

}  // namespace moe
