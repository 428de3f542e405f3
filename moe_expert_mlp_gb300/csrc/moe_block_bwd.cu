// Backward of the residual block's norms: the pre norm's gradient joined to
// the residual's, and the post norm's through gate, scale and norm -- both in
// one pass over the rows where a block's post norm and the next block's pre
// norm meet at the residual r'.
//
//   D   = s dres_in + N1^T(dx; r')             the gradient of r'
//   dy  = N2^T(b G (*) D; y)
//   N^T(dn; v): dxh = dn (*) (off + w)
//               dv  = rstd (dxh - [layer] mean(dxh) - xhat mean(dxh xhat))
//
// The statistics are taken again from r' and y, which the gradient reads
// anyway, instead of being kept from the forward.
//
// Bound by HBM.  The parameter gradients are sums over the tokens; every
// thread keeps its channels' sums in registers over all the rows of its
// group, a block joins its groups' sums in shared memory, and a second small
// kernel adds the blocks' partials in block order (no atomics: equal inputs
// give equal bits).  With a gate that does not depend on the token two sums
// carry every gradient of the post norm, S1 = sum_t D xhat and S0 = sum_t D:
//   dw = b G S1,  db = b G S0,  dG = b ((off + w) S1 + bias S0).
#include "moe_block.cuh"

namespace moe {
namespace {

template <int NV>
__device__ __forceinline__ float row_mean(const BlockArgs& p, Group& g, const float (&v)[NV][8]) {
  float s[1] = {0.0f};
#pragma unroll
  for (int u = 0; u < NV; ++u)
#pragma unroll
    for (int e = 0; e < 8; ++e) s[0] += v[u][e];
  group_sum(g, s);
  return s[0] / static_cast<float>(p.d);
}

template <typename TA, typename TR, int NV, bool PRE, bool POST, bool BIAS>
__global__ void __launch_bounds__(kBlockThreads, 1)
    k_block_bwd(const __grid_constant__ BlockArgs p) {
  constexpr int kSides = (PRE ? 1 : 0) + (POST ? 1 : 0);
  constexpr int kAcc = kSides * (BIAS ? 2 : 1);
  __shared__ float4 red[2 * kBlockThreads / 32];
  extern __shared__ float join[];                 // [kAcc][d], with several groups
  Group g = make_group(p, red);
  const int groups = blockDim.x / p.tpr;
  const float inv = 1.0f / static_cast<float>(p.d);
  UnitMap m[NV];
#pragma unroll
  for (int u = 0; u < NV; ++u) m[u] = unit_map(p, g.lane, u);
  float acc[kAcc][NV][8];
#pragma unroll
  for (int a = 0; a < kAcc; ++a)
#pragma unroll
    for (int u = 0; u < NV; ++u)
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[a][u][e] = 0.0f;

  for (int t = blockIdx.x * groups + g.id; t < p.T; t += gridDim.x * groups) {
    float D[NV][8];
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      if (p.dres_in.p != nullptr) {
        load_unit(row_ptr<const TR>(p.dres_in, t), m[u], p.vec, D[u]);
#pragma unroll
        for (int e = 0; e < 8; ++e) D[u][e] *= p.dres_scale;
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) D[u][e] = 0.0f;
      }
    }
    if constexpr (PRE) {
      float v[NV][8], dx[NV][8];
#pragma unroll
      for (int u = 0; u < NV; ++u) {
        load_unit(row_ptr<const TR>(p.res, t), m[u], p.vec, v[u]);
        load_unit(row_ptr<const TA>(p.dx, t), m[u], p.vec, dx[u]);
      }
      const bool layer = p.pre.kind == MOE_NORM_LAYER;
      if (layer) {
        const float mu = row_mean<NV>(p, g, v);
#pragma unroll
        for (int u = 0; u < NV; ++u)
#pragma unroll
          for (int e = 0; e < 8; ++e) v[u][e] = e < m[u].n ? v[u][e] - mu : 0.0f;
      }
      float s[3] = {0.0f, 0.0f, 0.0f};   // squares, dxh, dxh v
#pragma unroll
      for (int u = 0; u < NV; ++u) {
        float w[8];
        load_param(p.pre.w, p, m[u], p.pre.off, 1.0f, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float dxh = dx[u][e] * w[e];
          s[0] += v[u][e] * v[u][e];
          s[1] += dxh;
          s[2] += dxh * v[u][e];
        }
      }
      group_sum(g, s);
      const float rstd = 1.0f / sqrtf(s[0] * inv + p.pre.eps);
      const float m0 = layer ? s[1] * inv : 0.0f, m1 = s[2] * rstd * inv;
#pragma unroll
      for (int u = 0; u < NV; ++u) {
        float w[8];
        load_param(p.pre.w, p, m[u], p.pre.off, 1.0f, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float xh = v[u][e] * rstd;
          acc[0][u][e] += dx[u][e] * xh;
          if constexpr (BIAS) acc[1][u][e] += dx[u][e];
          if (e < m[u].n) D[u][e] += rstd * (dx[u][e] * w[e] - m0 - xh * m1);
        }
      }
    }
    if (p.dres.p != nullptr) {
#pragma unroll
      for (int u = 0; u < NV; ++u) store_unit(row_ptr<TR>(p.dres, t), m[u], p.vec, D[u]);
    }
    if constexpr (POST) {
      constexpr int kS1 = PRE ? (BIAS ? 2 : 1) : 0;
      float v[NV][8], wg[NV][8];                 // y - mu, (off + w) of each channel
#pragma unroll
      for (int u = 0; u < NV; ++u) load_unit(row_ptr<const TA>(p.y, t), m[u], p.vec, v[u]);
      const bool normed = p.post.kind != MOE_NORM_NONE;
      const bool layer = p.post.kind == MOE_NORM_LAYER;
      float rstd = 1.0f;
      if (layer) {
        const float mu = row_mean<NV>(p, g, v);
#pragma unroll
        for (int u = 0; u < NV; ++u)
#pragma unroll
          for (int e = 0; e < 8; ++e) v[u][e] = e < m[u].n ? v[u][e] - mu : 0.0f;
      }
      if (normed) {
        float q[1] = {0.0f};
#pragma unroll
        for (int u = 0; u < NV; ++u)
#pragma unroll
          for (int e = 0; e < 8; ++e) q[0] += v[u][e] * v[u][e];
        group_sum(g, q);
        rstd = 1.0f / sqrtf(q[0] * inv + p.post.eps);
      }
      float gt = 1.0f;
      if (p.gate == MOE_GATE_TOKEN)
        gt = gate_act(p.gate_act, *row_ptr<const float>(p.gate_rows, t));
      float s[3] = {0.0f, 0.0f, 0.0f};           // dxh, dxh xhat, D n
#pragma unroll
      for (int u = 0; u < NV; ++u) {
        float b[8], gv[8], gs[8];
        load_param(p.post.w, p, m[u], p.post.off, 1.0f, wg[u]);
        load_param(p.post.b, p, m[u], 0.0f, 0.0f, b);
        if (p.gate == MOE_GATE_CHANNEL)
          load_param(p.gate_rows.p, p, m[u], 0.0f, 1.0f, gv);
        else if (p.gate == MOE_GATE_FULL)
          load_unit(row_ptr<const TA>(p.gate_rows, t), m[u], p.vec, gv);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          gv[e] = p.gate == MOE_GATE_CHANNEL || p.gate == MOE_GATE_FULL ? gate_act(p.gate_act, gv[e])
                                                                       : gt;
          gs[e] = gate_slope(p.gate_act, gv[e]);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float xh = v[u][e] * rstd;
          const float n = xh * wg[u][e] + b[e];
          const float Dn = D[u][e] * n;
          if (p.gate == MOE_GATE_FULL) gs[e] *= p.branch_scale * Dn;
          // the gate joins the sums where it differs from token to token
          const float q = p.gate == MOE_GATE_TOKEN || p.gate == MOE_GATE_FULL ? D[u][e] * gv[e]
                                                                            : D[u][e];
          acc[kS1][u][e] += q * xh;
          if constexpr (BIAS) acc[kS1 + 1][u][e] += q;
          s[2] += Dn;
          D[u][e] = p.branch_scale * gv[e] * D[u][e] * wg[u][e];   // dxh
          s[0] += D[u][e];
          s[1] += D[u][e] * xh;
        }
        if (p.gate == MOE_GATE_FULL && p.dgate.p != nullptr)
          store_unit(row_ptr<TA>(p.dgate, t), m[u], p.vec, gs);
      }
      if (normed || p.gate == MOE_GATE_TOKEN) group_sum(g, s);
      if (p.gate == MOE_GATE_TOKEN && p.dgate.p != nullptr && g.lane == 0)
        *row_ptr<float>(p.dgate, t) = p.branch_scale * s[2] * gate_slope(p.gate_act, gt);
      if (normed) {
        const float m0 = layer ? s[0] * inv : 0.0f, m1 = s[1] * inv;
#pragma unroll
        for (int u = 0; u < NV; ++u)
#pragma unroll
          for (int e = 0; e < 8; ++e) D[u][e] = rstd * (D[u][e] - m0 - v[u][e] * rstd * m1);
      }
#pragma unroll
      for (int u = 0; u < NV; ++u) store_unit(row_ptr<TA>(p.dy, t), m[u], p.vec, D[u]);
    }
  }

  // the block's sums: its groups one after another
  float* part = p.part + static_cast<long long>(blockIdx.x) * kAcc * p.d;
  for (int i = 0; i < groups; ++i) {
    if (i > 0) __syncthreads();
    if (g.id != i) continue;
    float* to = i + 1 == groups ? part : join;
#pragma unroll
    for (int a = 0; a < kAcc; ++a)
#pragma unroll
      for (int u = 0; u < NV; ++u)
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (e < m[u].n) {
            const int c = m[u].c0 + e * m[u].step;
            const float before = i > 0 ? join[a * p.d + c] : 0.0f;
            to[a * p.d + c] = before + acc[a][u][e];
          }
  }
}

// Adds the blocks' partials channel by channel, and turns the sums into the
// parameters' gradients.  32 channels a block, 8 rows of partials at a time.
__global__ void __launch_bounds__(256) k_block_bwd_finish(const __grid_constant__ BlockArgs p,
                                                          const __grid_constant__ BlockGrads o) {
  __shared__ float sums[4][8][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  for (int a = 0; a < o.acc; ++a) {
    float s = 0.0f;
    if (c < p.d)
      for (int i = warp; i < o.parts; i += 8)
        s += p.part[(static_cast<long long>(i) * o.acc + a) * p.d + c];
    sums[a][warp][lane] = s;
  }
  __syncthreads();
  if (warp != 0 || c >= p.d) return;
  float S[4];
  for (int a = 0; a < o.acc; ++a) {
    S[a] = 0.0f;
    for (int i = 0; i < 8; ++i) S[a] += sums[a][i][lane];
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

template <typename TA, typename TR, int NV, bool PRE, bool POST>
cudaError_t launch_sides(const BlockArgs& a, bool bias, int blocks, int threads, size_t smem,
                         cudaStream_t s) {
  if (bias)
    k_block_bwd<TA, TR, NV, PRE, POST, true><<<blocks, threads, smem, s>>>(a);
  else
    k_block_bwd<TA, TR, NV, PRE, POST, false><<<blocks, threads, smem, s>>>(a);
  return cudaGetLastError();
}

template <typename TA, typename TR, int NV>
cudaError_t launch_nv(const BlockArgs& a, const BlockGrads& o, int blocks, int threads,
                      size_t smem, cudaStream_t s) {
  if (o.pre && o.post) return launch_sides<TA, TR, NV, true, true>(a, o.bias, blocks, threads, smem, s);
  if (o.pre) return launch_sides<TA, TR, NV, true, false>(a, o.bias, blocks, threads, smem, s);
  return launch_sides<TA, TR, NV, false, true>(a, o.bias, blocks, threads, smem, s);
}

template <typename TA, typename TR>
cudaError_t launch_types(const BlockArgs& a, const BlockGrads& o, int blocks, int threads,
                         size_t smem, cudaStream_t s) {
  if (a.nv == 1) return launch_nv<TA, TR, 1>(a, o, blocks, threads, smem, s);
  if (a.nv == 2) return launch_nv<TA, TR, 2>(a, o, blocks, threads, smem, s);
  return launch_nv<TA, TR, 4>(a, o, blocks, threads, smem, s);
}

}  // namespace

cudaError_t launch_block_bwd(const BlockArgs& a, BlockGrads o, int dtype, int res_dtype, int sms,
                             cudaStream_t s) {
  const int groups = kBlockThreads / a.tpr, threads = groups * a.tpr;
  o.acc = (o.pre + o.post) * (o.bias ? 2 : 1);
  o.parts = min((a.T + groups - 1) / groups, min(sms, kBlockBwdMaxParts));
  const size_t smem = groups > 1 ? static_cast<size_t>(o.acc) * a.d * sizeof(float) : 0;
  cudaError_t e = cudaSuccess;
  if (o.parts > 0) {
    if (dtype == MOE_DTYPE_FP32)
      e = launch_types<float, float>(a, o, o.parts, threads, smem, s);
    else if (res_dtype == MOE_DTYPE_FP32)
      e = launch_types<__nv_bfloat16, float>(a, o, o.parts, threads, smem, s);
    else
      e = launch_types<__nv_bfloat16, __nv_bfloat16>(a, o, o.parts, threads, smem, s);
  }
  const bool any = o.dpre_w || o.dpre_b || o.dpost_w || o.dpost_b || o.dgate;
  if (e == cudaSuccess && any) {
    k_block_bwd_finish<<<(a.d + 31) / 32, 256, 0, s>>>(a, o);
    e = cudaGetLastError();
  }
  return e;
}

}  // namespace moe
