// Backward kernel of the residual block's norms: the pre norm's gradient joined
// to the residual's, and the post norm's through gate, scale and norm -- both in
// one pass over the rows where a block's post norm and the next block's pre
// norm meet at the residual r'.  Instantiated type by type in
// moe_block_bwd_*.cu.
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
// kernel (moe_block_bwd.cu) adds the blocks' partials in block order (no
// atomics: equal inputs give equal bits).  With a gate that does not depend on
// the token two sums carry every gradient of the post norm, S1 = sum_t D xhat
// and S0 = sum_t D:
//   dw = b G S1,  db = b G S0,  dG = b ((off + w) S1 + bias S0).
//
// The sums' registers leave room for one block of up to 512 threads on an SM,
// so nothing but the block itself hides its loads: each thread copies its own
// 16-byte pieces of the next rows into its own places of a ring in shared
// memory (cp.async), and waits for no one else's.
#pragma once

#include "moe_block.cuh"

namespace moe {
namespace {

__device__ __forceinline__ void copy16_async(void* to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(to)), "l"(from)
               : "memory");
}
__device__ __forceinline__ void copies_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// One row tensor of a row: a thread's units, in its places of the ring (VEC)
// or in registers.
template <typename T, int NV, bool VEC>
struct RowPart {
  static constexpr int kPieces = VEC ? NV * static_cast<int>(sizeof(T)) / 2 : 0;
  Raw<T, VEC> held[VEC ? 1 : NV];
  uint4* at;   // piece i at at[i * threads]

  __device__ __forceinline__ void copy(const T* row, const Unit<VEC> (&m)[NV], int threads) {
    if constexpr (VEC) {
      constexpr int kHalves = sizeof(T) / 2;
#pragma unroll
      for (int u = 0; u < NV; ++u)
        if (m[u].has(0)) {
#pragma unroll
          for (int h = 0; h < kHalves; ++h)
            copy16_async(at + (u * kHalves + h) * threads,
                         reinterpret_cast<const uint4*>(row + m[u].c0) + h);
        }
    }
  }
  __device__ __forceinline__ void fetch(const T* row, const Unit<VEC> (&m)[NV]) {
    if constexpr (!VEC) {
#pragma unroll
      for (int u = 0; u < NV; ++u) held[u].template load<true>(row, m[u]);
    }
  }
  __device__ __forceinline__ Raw<T, VEC> get(const Unit<VEC>& m, int u, int threads) const {
    if constexpr (VEC) {
      constexpr int kHalves = sizeof(T) / 2;
      Raw<T, VEC> r;
#pragma unroll
      for (int h = 0; h < kHalves; ++h) {
        uint4 q = make_uint4(0, 0, 0, 0);
        if (m.has(0)) q = at[(u * kHalves + h) * threads];
        r.w[4 * h] = q.x, r.w[4 * h + 1] = q.y, r.w[4 * h + 2] = q.z, r.w[4 * h + 3] = q.w;
      }
      return r;
    } else {
      return held[u];
    }
  }
};

// Weights of a thread's units: in registers where they fit, else from L1.
template <int NV, bool VEC, bool HELD>
struct Weights {
  float held[HELD ? NV : 1][8];
  template <typename F>
  __device__ __forceinline__ void fetch(F&& make) {
    if constexpr (HELD) {
#pragma unroll
      for (int u = 0; u < NV; ++u) make(u, held[u]);
    }
  }
  template <typename F>
  __device__ __forceinline__ void get(F&& make, int u, float (&v)[8]) const {
    if constexpr (HELD) {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = held[u][e];
    } else {
      make(u, v);
    }
  }
};

constexpr int kRing = 3;   // rows of a group in the ring, at most

// Pieces of a ring row: the tensors that the kernel copies.
template <typename TA, typename TR, int NV, bool VEC, bool PRE, bool POST>
__host__ __device__ constexpr int ring_pieces() {
  return RowPart<TR, NV, VEC>::kPieces * (PRE ? 2 : 1) +
         RowPart<TA, NV, VEC>::kPieces * ((PRE ? 1 : 0) + (POST ? 1 : 0));
}

template <typename TA, typename TR, int NV, bool VEC, bool PRE, bool POST, bool BIAS>
__global__ void __launch_bounds__(kBlockThreads, 1)
    k_block_bwd(const __grid_constant__ BlockArgs p, int ring) {
  constexpr int kSides = (PRE ? 1 : 0) + (POST ? 1 : 0);
  constexpr int kAcc = kSides * (BIAS ? 2 : 1);
  constexpr int kS1 = PRE ? (BIAS ? 2 : 1) : 0;        // the post norm's first sum
  constexpr bool kHeld = NV == 1 || (NV == 2 && !BIAS);
  constexpr int kPieces = ring_pieces<TA, TR, NV, VEC, PRE, POST>();
  __shared__ float4 red[2 * kBlockThreads / 32];
  extern __shared__ uint4 dyn[];                 // the ring; then the groups' sums
  Group g = make_group(p, red);
  const int groups = blockDim.x / p.tpr, threads = blockDim.x;
  const float inv = 1.0f / static_cast<float>(p.d);
  const bool pre_layer = PRE && p.pre.kind == MOE_NORM_LAYER;
  const bool normed = POST && p.post.kind != MOE_NORM_NONE;
  const bool post_layer = POST && p.post.kind == MOE_NORM_LAYER;
  const bool full = p.gate == MOE_GATE_FULL, token = p.gate == MOE_GATE_TOKEN;
  Unit<VEC> m[NV];
#pragma unroll
  for (int u = 0; u < NV; ++u) m[u] = Unit<VEC>(p, g.lane, u);

  // the ring's places of this thread, and the copy of row t into slot i
  RowPart<TR, NV, VEC> dres_in, res;
  RowPart<TA, NV, VEC> dx, y;
  auto place = [&](int slot) {
    if constexpr (VEC) {
      uint4* at = dyn + static_cast<size_t>(slot) * kPieces * threads + threadIdx.x;
      dres_in.at = at;
      at += RowPart<TR, NV, VEC>::kPieces * threads;
      if constexpr (PRE) {
        res.at = at;
        at += RowPart<TR, NV, VEC>::kPieces * threads;
        dx.at = at;
        at += RowPart<TA, NV, VEC>::kPieces * threads;
      }
      y.at = at;
    }
  };
  auto copy = [&](int t, int slot) {
    if constexpr (VEC) {
      if (t < p.T) {
        place(slot);
        if constexpr (PRE) {
          res.copy(row_ptr<const TR>(p.res, t), m, threads);
          dx.copy(row_ptr<const TA>(p.dx, t), m, threads);
        }
        if constexpr (POST) y.copy(row_ptr<const TA>(p.y, t), m, threads);
        if (p.dres_in.p != nullptr) dres_in.copy(row_ptr<const TR>(p.dres_in, t), m, threads);
      }
      copies_commit();   // one group a row, empty past the end
    }
  };

  const int step = gridDim.x * groups;
  int t = blockIdx.x * groups + g.id;
  for (int i = 0; i < ring; ++i) copy(t + i * step, i);

  // the pre norm's weights, and the post norm's times gate and scale where
  // neither changes from token to token
  auto pre_weight = [&](int u, float (&v)[8]) { load_param(p.pre.w, p, m[u], p.pre.off, 1.0f, v); };
  auto post_weight = [&](int u, float (&v)[8]) {
    load_param(p.post.w, p, m[u], p.post.off, 1.0f, v);
    if (p.gate == MOE_GATE_CHANNEL) {
      float q[8];
      load_param(p.gate_rows.p, p, m[u], 0.0f, 1.0f, q);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] *= p.branch_scale * gate_act(p.gate_act, q[e]);
    } else if (p.gate == MOE_GATE_NONE) {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] *= p.branch_scale;
    }
  };
  Weights<NV, VEC, kHeld> w1, w2;
  if constexpr (PRE) w1.fetch(pre_weight);
  if constexpr (POST) w2.fetch(post_weight);

  float acc[kAcc][NV][8];
#pragma unroll
  for (int a = 0; a < kAcc; ++a)
#pragma unroll
    for (int u = 0; u < NV; ++u)
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[a][u][e] = 0.0f;

  int slot = 0;
  for (; t < p.T; t += step) {
    if constexpr (VEC) {
      if (ring == 3) copies_wait<2>();
      else if (ring == 2) copies_wait<1>();
      else copies_wait<0>();
      place(slot);
    } else {
      if constexpr (PRE) {
        res.fetch(row_ptr<const TR>(p.res, t), m);
        dx.fetch(row_ptr<const TA>(p.dx, t), m);
      }
      if constexpr (POST) y.fetch(row_ptr<const TA>(p.y, t), m);
      if (p.dres_in.p != nullptr) dres_in.fetch(row_ptr<const TR>(p.dres_in, t), m);
    }
    float gt = 1.0f;                             // the token's gate
    if (token) gt = gate_act(p.gate_act, *row_ptr<const float>(p.gate_rows, t));
    float mu1 = 0.0f, mu2 = 0.0f;
    if (pre_layer || post_layer) {
      float s[2] = {0.0f, 0.0f};
#pragma unroll
      for (int u = 0; u < NV; ++u) {
        if constexpr (PRE) {
          const Raw<TR, VEC> a = res.get(m[u], u, threads);
#pragma unroll
          for (int e = 0; e < 8; ++e) s[0] += a.get(e);
        }
        if constexpr (POST) {
          const Raw<TA, VEC> a = y.get(m[u], u, threads);
#pragma unroll
          for (int e = 0; e < 8; ++e) s[1] += a.get(e);
        }
      }
      group_sum(g, s);
      if (pre_layer) mu1 = s[0] * inv;
      if (post_layer) mu2 = s[1] * inv;
    }

    // Sums over the row.  With a pre norm: its squares, dxh, dxh v and the
    // post norm's squares; without: the post norm's own, as D is known.
    float D[NV][8];
    float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    auto load_D = [&](int u) {
      if (p.dres_in.p != nullptr) {
        const Raw<TR, VEC> a = dres_in.get(m[u], u, threads);
#pragma unroll
        for (int e = 0; e < 8; ++e) D[u][e] = p.dres_scale * a.get(e);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) D[u][e] = 0.0f;
      }
    };
    // the post norm's sums of unit u: dxh, dxh (y - mu), D bias; dxh without
    // the token's gate (and without the scale where there is a token or full
    // gate), which the caller applies to the sums
    auto post_sums = [&](int u, float& s1, float& s2, float& s3) {
      const Raw<TA, VEC> a = y.get(m[u], u, threads);
      float w[8];
      w2.get(post_weight, u, w);
      if (full) {
        float q[8];
        load_row(row_ptr<const TA>(p.gate_rows, t), m[u], q);
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] *= gate_act(p.gate_act, q[e]);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float dxh = D[u][e] * w[e];
        s1 += dxh;
        s2 += dxh * (a.get(e) - mu2);            // D is 0 past the row's end
      }
      if (token && p.post.b != nullptr) {
        float b[8];
        load_param(p.post.b, p, m[u], 0.0f, 0.0f, b);
#pragma unroll
        for (int e = 0; e < 8; ++e) s3 += D[u][e] * b[e];
      }
    };
    auto post_squares = [&](int u, float& q) {
      const Raw<TA, VEC> a = y.get(m[u], u, threads);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float c = !post_layer || m[u].has(e) ? a.get(e) - mu2 : 0.0f;
        q += c * c;
      }
    };
    float rstd2 = 1.0f;
    if constexpr (PRE) {
#pragma unroll
      for (int u = 0; u < NV; ++u) {
        const Raw<TR, VEC> a = res.get(m[u], u, threads);
        const Raw<TA, VEC> b = dx.get(m[u], u, threads);
        float w[8];
        w1.get(pre_weight, u, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float c = !pre_layer || m[u].has(e) ? a.get(e) - mu1 : 0.0f;
          const float dxh = b.get(e) * w[e];
          s[0] += c * c;
          s[1] += dxh;
          s[2] += dxh * c;
        }
        if (normed) post_squares(u, s[3]);
      }
      group_sum(g, s);
      const float rstd = 1.0f / sqrtf(s[0] * inv + p.pre.eps);
      const float m0 = pre_layer ? s[1] * inv : 0.0f, m1 = s[2] * rstd * inv;
      if (normed) rstd2 = 1.0f / sqrtf(s[3] * inv + p.post.eps);
#pragma unroll
      for (int u = 0; u < NV; ++u) {
        load_D(u);
        const Raw<TR, VEC> a = res.get(m[u], u, threads);
        const Raw<TA, VEC> b = dx.get(m[u], u, threads);
        float w[8];
        w1.get(pre_weight, u, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float xh = (a.get(e) - mu1) * rstd;
          acc[0][u][e] += b.get(e) * xh;         // dx is 0 past the row's end
          if constexpr (BIAS) acc[1][u][e] += b.get(e);
          D[u][e] += m[u].has(e) ? rstd * (b.get(e) * w[e] - m0 - xh * m1) : 0.0f;
        }
        if (p.dres.p != nullptr) store_unit(row_ptr<TR>(p.dres, t), m[u], D[u]);
      }
    } else {
#pragma unroll
      for (int u = 0; u < NV; ++u) {
        load_D(u);
        if (p.dres.p != nullptr) store_unit(row_ptr<TR>(p.dres, t), m[u], D[u]);
      }
    }

    if constexpr (POST) {
      float e1, e2, e3;
      if constexpr (PRE) {
        float q[3] = {0.0f, 0.0f, 0.0f};
        if (normed || token) {
#pragma unroll
          for (int u = 0; u < NV; ++u) post_sums(u, q[0], q[1], q[2]);
          group_sum(g, q);
        }
        e1 = q[0], e2 = q[1], e3 = q[2];
      } else {
        if (normed || token) {
#pragma unroll
          for (int u = 0; u < NV; ++u) {
            post_sums(u, s[1], s[2], s[3]);
            if (normed) post_squares(u, s[0]);
          }
          group_sum(g, s);
        }
        if (normed) rstd2 = 1.0f / sqrtf(s[0] * inv + p.post.eps);
        e1 = s[1], e2 = s[2], e3 = s[3];
      }
      if (token && p.dgate.p != nullptr && g.lane == 0)
        *row_ptr<float>(p.dgate, t) =
            p.branch_scale * (rstd2 * e2 + e3) * gate_slope(p.gate_act, gt);
      const float scale = token ? p.branch_scale * gt : full ? p.branch_scale : 1.0f;
      const float m0 = post_layer ? scale * e1 * inv : 0.0f;
      const float m1 = normed ? scale * e2 * rstd2 * inv : 0.0f;
      const float out = normed ? rstd2 : 1.0f;
#pragma unroll
      for (int u = 0; u < NV; ++u) {
        const Raw<TA, VEC> a = y.get(m[u], u, threads);
        float w[8], dy[8];
        w2.get(post_weight, u, w);
        if (full) {
          float q[8], dg[8], b[8];
          load_row(row_ptr<const TA>(p.gate_rows, t), m[u], q);
          load_param(p.post.b, p, m[u], 0.0f, 0.0f, b);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float gv = gate_act(p.gate_act, q[e]);
            const float n = (a.get(e) - mu2) * rstd2 * w[e] + b[e];
            dg[e] = p.branch_scale * D[u][e] * n * gate_slope(p.gate_act, gv);
            D[u][e] *= gv;                       // the gate joins the sums
          }
          if (p.dgate.p != nullptr) store_unit(row_ptr<TA>(p.dgate, t), m[u], dg);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float xh = (a.get(e) - mu2) * rstd2;
          const float q = token ? D[u][e] * gt : D[u][e];
          acc[kS1][u][e] += q * xh;              // D is 0 past the row's end
          if constexpr (BIAS) acc[kS1 + 1][u][e] += q;
          dy[e] = out * (scale * D[u][e] * w[e] - m0 - xh * m1);
        }
        store_unit(row_ptr<TA>(p.dy, t), m[u], dy);
      }
    }
    copy(t + ring * step, slot);
    slot = slot + 1 == ring ? 0 : slot + 1;
  }

  // the block's sums: its groups one after another
  if constexpr (VEC) copies_wait<0>();
  float* join = reinterpret_cast<float*>(dyn);   // [kAcc][d], with several groups
  float* part = p.part + static_cast<long long>(blockIdx.x) * kAcc * p.d;
  if (groups > 1) __syncthreads();               // the ring is read no more
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
          if (m[u].has(e)) {
            const int c = m[u].at(e);
            const float before = i > 0 ? join[a * p.d + c] : 0.0f;
            to[a * p.d + c] = before + acc[a][u][e];
          }
  }
}

constexpr size_t kBlockSmem = 220 * 1024;   // shared memory the ring may take

template <typename TA, typename TR, int NV, bool VEC, bool PRE, bool POST, bool BIAS>
cudaError_t launch_kernel(const BlockArgs& a, int blocks, int groups, cudaStream_t s) {
  const int threads = groups * a.tpr;
  if constexpr (VEC && NV == 4) {
    // the widest fp32 rows: not one fits the ring
    if (static_cast<size_t>(ring_pieces<TA, TR, NV, VEC, PRE, POST>()) * threads * 16 > kBlockSmem)
      return launch_kernel<TA, TR, NV, false, PRE, POST, BIAS>(a, blocks, groups, s);
  }
  constexpr int kAcc = ((PRE ? 1 : 0) + (POST ? 1 : 0)) * (BIAS ? 2 : 1);
  size_t row = static_cast<size_t>(ring_pieces<TA, TR, NV, VEC, PRE, POST>()) * threads * 16;
  int ring = row == 0 ? 0 : static_cast<int>(kBlockSmem / row);
  if (ring > kRing) ring = kRing;
  size_t smem = ring * row;
  if (groups > 1) {
    const size_t join = static_cast<size_t>(kAcc) * a.d * sizeof(float);
    if (join > smem) smem = join;
  }
  auto* k = k_block_bwd<TA, TR, NV, VEC, PRE, POST, BIAS>;
  if (smem > 32 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(smem));
    if (e != cudaSuccess) return e;
  }
  k<<<blocks, threads, smem, s>>>(a, ring);
  return cudaGetLastError();
}

template <typename TA, typename TR, int NV, bool VEC>
cudaError_t launch_nv(const BlockArgs& a, const BlockGrads& o, int groups, cudaStream_t s) {
  if (o.pre && o.post)
    return o.bias ? launch_kernel<TA, TR, NV, VEC, true, true, true>(a, o.parts, groups, s)
                  : launch_kernel<TA, TR, NV, VEC, true, true, false>(a, o.parts, groups, s);
  if (o.pre)
    return o.bias ? launch_kernel<TA, TR, NV, VEC, true, false, true>(a, o.parts, groups, s)
                  : launch_kernel<TA, TR, NV, VEC, true, false, false>(a, o.parts, groups, s);
  return o.bias ? launch_kernel<TA, TR, NV, VEC, false, true, true>(a, o.parts, groups, s)
                : launch_kernel<TA, TR, NV, VEC, false, true, false>(a, o.parts, groups, s);
}

}  // namespace

template <typename TA, typename TR>
cudaError_t launch_block_bwd_types(BlockArgs a, BlockGrads& o, int sms, cudaStream_t s) {
  // the fewest units a thread (1, 2 or 4) with which 512 threads hold a row
  const int units = (a.d + kUnit - 1) / kUnit;
  const int nv = units <= kBlockThreads ? 1 : units <= 2 * kBlockThreads ? 2 : 4;
  a.tpr = ((units + nv - 1) / nv + 31) / 32 * 32;
  const int groups = kBlockThreads / a.tpr;
  o.parts = (a.T + groups - 1) / groups;
  if (o.parts > sms) o.parts = sms;
  if (o.parts > kBlockBwdMaxParts) o.parts = kBlockBwdMaxParts;
  if (o.parts == 0) return cudaSuccess;
  if (a.vec) {
    if (nv == 1) return launch_nv<TA, TR, 1, true>(a, o, groups, s);
    if (nv == 2) return launch_nv<TA, TR, 2, true>(a, o, groups, s);
    return launch_nv<TA, TR, 4, true>(a, o, groups, s);
  }
  if (nv == 1) return launch_nv<TA, TR, 1, false>(a, o, groups, s);
  if (nv == 2) return launch_nv<TA, TR, 2, false>(a, o, groups, s);
  return launch_nv<TA, TR, 4, false>(a, o, groups, s);
}

}  // namespace moe
