// Forward kernel of the residual block's norms: the pre norm x = N1(r), and
// the post norm r' = a r + b G (*) N2(y) with the next block's norm
// x' = N1(r') in the same pass, y read as rows or combined from the routed
// expert rows.  Instantiated type by type in moe_block_fwd_*.cu.
//
// Bound by HBM: a few operations a channel against 4 to 16 bytes.  A row is
// read once, its sums are taken from registers, and what follows from them is
// stored.
//
// Many aligned rows: one block of up to 512 threads an SM (k_block_fwd_ring),
// whose groups walk down the rows with their parameters in registers, while
// each thread copies its own 16-byte pieces of the rows to come into its own
// places of a ring in shared memory (cp.async) and waits for no one else's (an
// fp32 warp: for its own threads').  Measured: post norm with the next norm,
// 16384 x 7168 over an fp32 residual, 218 us = 6.5 TB/s, 95 % of the rate of a
// copy, all in bf16 165 us = 5.7 TB/s; on expert rows, 16384 x 2880, k = 4, 136 us = 5.6 TB/s (the ring holds
// one token's rows there, so a group's loads and sums do not overlap, only the
// five groups'); pre layer norm, 4096 x 2048, 9.4 us = 3.6 TB/s, of which about
// 3 us are the first rows' way in and the last ones' out; RMS, 16384 x 4096,
// 48 us = 5.5 TB/s.  The general form takes two or three sums a row one after
// another: both layer norms with biases and a channel gate, 16384 x 7168, 234 us
// = 4.0 TB/s; with a gate tensor, read past the ring, 395 us = 3.0 TB/s.
//
// Few rows, rows that are not aligned, and tokens whose expert rows do not fit
// the ring: one group a row (k_block_fwd).  With
// few rows nothing hides a row's latency, so the group is as large as the row
// allows and the parameters are fetched together with the row instead of after
// its sums.
#pragma once

#include "moe_block.cuh"

namespace moe {
namespace {

// Statistics of the row held in v: mean (layer norm) and 1/sqrt(. + eps).
// The layer norm's variance sums squares about the mean, from registers.
template <int NV, bool VEC>
__device__ __forceinline__ void row_stats(const BlockArgs& p, const BlockNorm& n, Group<false>& g,
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
  rstd = rsqrtf(q[0] * inv + n.eps);
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
__device__ __forceinline__ void normalize(const BlockArgs& p, const BlockNorm& n, Group<false>& g,
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
__device__ __forceinline__ void combine_rows(const BlockArgs& p, int t, const Group<false>& g,
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

// Blocks that have to fit an SM.  Rows that are not aligned wait for many small
// loads: with bf16 branches four blocks of 64 registers hide more of it than two
// without spills (routed, k = 6, 4096 x 2047: 117 and 174 us; post norm,
// 929 x 3361: 17 and 22), with fp32 ones and for the pre norm they do not
// (routed, 4096 x 1441: 82 and 69 us; pre norm, 4096 x 2047: 16.2 and 15.7).
template <typename TA, int NV, bool VEC, int MODE>
constexpr int kResidentFwd = !VEC && NV == 2 && MODE != kPre && sizeof(TA) == 2 ? 4 : 1;

template <typename TA, typename TR, int NV, bool VEC, int MODE, bool HOIST>
__global__ void __launch_bounds__(HOIST ? kBlockThreads : kBlockThreads / 2,
                                  kResidentFwd<TA, NV, VEC, MODE>)
    k_block_fwd(const __grid_constant__ BlockArgs p) {
  __shared__ float red[kRedFloats];
  Group<false> g = make_group<false>(p, red);
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

// The routed branch's rows of a token, prefetched by lane: lane s of a warp
// holds slot s's row (-1: not a row) and weight.
struct Slots {
  int row;
  float w;
  __device__ __forceinline__ void load(const BlockArgs& p, int t, int lane) {
    const int s = lane & 31;
    row = -1;
    w = 0.0f;
    if (t < p.T && s < p.k) {
      const long long at = static_cast<long long>(t) * p.k + s;
      row = __ldg(p.row_of + at);
      w = __ldg(p.topk_w + at);
      if (row < 0 || row >= p.capacity) {
        if (lane < 32) atomicOr(p.status, MOE_DEV_BAD_OFFSETS);
        row = -1;
      }
    }
  }
};

template <typename TA, typename TR, int NV, int MODE, bool BIAS, bool PLAIN>
__global__ void __launch_bounds__(kBlockThreads, 1)
    k_block_fwd_ring(const __grid_constant__ BlockArgs p, int ring) {
  constexpr bool kHeld = NV <= 2 || PLAIN;
  using Res = RowPart<TR, NV, true>;
  using Act = RowPart<TA, NV, true>;
  __shared__ float red[kRedFloats];
  extern __shared__ uint4 dyn[];
  Group<true> g = make_group<true>(p, red);
  const int groups = blockDim.x / p.tpr;
  const float inv = 1.0f / static_cast<float>(p.d);
  const bool full = !PLAIN && p.gate == MOE_GATE_FULL, token = p.gate == MOE_GATE_TOKEN;
  const int slots = MODE == kRouted ? p.k : MODE == kPost ? 1 : 0;
  const int pieces = Res::kPieces + slots * Act::kPieces;
  Unit<true> m[NV];
#pragma unroll
  for (int u = 0; u < NV; ++u) m[u] = Unit<true>(p, g.lane, u);

  const int step = gridDim.x * groups;
  int t = blockIdx.x * groups + g.id;
  Res res;
  Act y;
  auto place = [&](int slot) {
    res.at = dyn + slot * pieces * kBlockThreads;
    y.at = res.at + Res::kPlaces;
  };
  // copies row t (its expert rows given by s) into a slot of the ring
  auto copy = [&](int row, int slot, const Slots& s) {
    if (row < p.T) {
      place(slot);
      if constexpr (MODE == kPost) y.copy(row_ptr<const TA>(p.y, row), m);
      if constexpr (MODE == kRouted) {
        for (int i = 0; i < slots; ++i) {
          const int r = __shfl_sync(0xFFFFFFFFu, s.row, i);
          if (r >= 0) y.copy(row16<const TA>(p.y, r), m);
          y.at += Act::kPlaces;
        }
      }
      // (the 64-bit product here, the wide one for the expert rows, by
      // measurement: post norm, 16384 x 7168 over an fp32 residual, 222 and 241 us;
      // routed, 16384 x 2880, k = 4, 145 and 134)
      res.copy(MODE == kRouted ? row16<const TR>(p.res, row) : row_ptr<const TR>(p.res, row), m);
    }
    copies_commit();   // one group a row, empty past the end
  };
  // routed: now, the rows in the ring behind it, and the one to copy next
  Slots s0, s1, s2, next;
  if constexpr (MODE == kRouted) {
    s0.load(p, t, g.lane);
    s1.load(p, t + step, g.lane);
    s2.load(p, t + 2 * step, g.lane);
    next.load(p, t + ring * step, g.lane);
  }
  copy(t, 0, s0);
  if (ring > 1) copy(t + step, 1, s1);
  if (ring > 2) copy(t + 2 * step, 2, s2);

  // the parameters; the post norm's times gate and scale where neither changes
  // from token to token
  auto scaled = [&](int u, F2 (&v)[4]) {
    if (p.gate == MOE_GATE_CHANNEL) {
      F2 q[4];
      load_param(p.gate_rows.p, p, m[u], 0.0f, 1.0f, q);
      gate_unit(p.gate_act, q);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = v[i] * q[i];
    }
    if (!full && !token) {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = v[i] * f2(p.branch_scale);
    }
  };
  auto post_weight = [&](int u, F2 (&v)[4]) {
    load_param(p.post.w, p, m[u], p.post.off, 1.0f, v);
    scaled(u, v);
  };
  auto post_bias = [&](int u, F2 (&v)[4]) {
    load_param(p.post.b, p, m[u], 0.0f, 0.0f, v);
    scaled(u, v);
  };
  auto pre_weight = [&](int u, F2 (&v)[4]) { load_param(p.pre.w, p, m[u], p.pre.off, 1.0f, v); };
  auto pre_bias = [&](int u, F2 (&v)[4]) { load_param(p.pre.b, p, m[u], 0.0f, 0.0f, v); };
  Weights<NV, kHeld> w1, w2;
  Weights<NV, kHeld && BIAS> b1, b2;
  if constexpr (MODE != kPre) {
    w2.fetch(post_weight);
    if constexpr (BIAS) b2.fetch(post_bias);
  }
  if (p.x.p != nullptr) {
    w1.fetch(pre_weight);
    if constexpr (BIAS) b1.fetch(pre_bias);
  }

  const F2 zero = f2(0.0f);
  F2 v[NV][4];
  // mean and 1/sqrt(. + eps) of the row in v
  auto stats = [&](const BlockNorm& n, float& mu, float& rstd) {
    mu = 0.0f;
    if (!PLAIN && n.kind == MOE_NORM_LAYER) {
      F2 a = zero;
#pragma unroll
      for (int u = 0; u < NV; ++u) {
        if (beyond(m[u])) continue;
#pragma unroll
        for (int i = 0; i < 4; ++i) a = a + v[u][i];
      }
      float s[1] = {sum(a)};
      group_sum(g, s);
      mu = s[0] * inv;
    }
    F2 a = zero;
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      if (beyond(m[u])) continue;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const F2 c = PLAIN ? v[u][i] : v[u][i] + f2(-mu);
        a = fma2(c, c, a);
      }
    }
    float s[1] = {sum(a)};
    group_sum(g, s);
    rstd = rsqrtf(s[0] * inv + n.eps);
  };

  float next_gate = token_gate(p, t);
  int slot = 0;
  constexpr bool kPipe = MODE == kPost && PLAIN;
  if constexpr (kPipe) {
    // The squares of this row's r' and of the next row's y meet in one sum, so
    // that a row waits once.
    float s[2];                                  // r', y of the row behind
    auto next_squares = [&]() {
      F2 a = zero;
#pragma unroll
      for (int u = 0; u < NV; ++u) {
        if (beyond(m[u])) continue;
        const Raw<TA, true> q = y.get(u);
#pragma unroll
        for (int i = 0; i < 4; ++i) a = fma2(q.pair(i), q.pair(i), a);
      }
      s[1] = sum(a);
    };
    if (t < p.T) {
      ring_wait(ring);
      place(0);
      next_squares();
      s[0] = 0.0f;
      group_sum(g, s);
    }
    for (; t < p.T; t += step) {
      const float gt = token ? gate_act(p.gate_act, next_gate) : 1.0f;
      next_gate = token_gate(p, t + step);
      place(slot);
      const float rstd = rsqrtf(s[1] * inv + p.post.eps);
      const F2 k1 = f2(rstd * (token ? p.branch_scale * gt : 1.0f)), a1 = f2(p.res_scale);
      F2 sq = zero;
#pragma unroll
      for (int u = 0; u < NV; ++u) {
        if (beyond(m[u])) continue;
        const Raw<TA, true> q = y.get(u);
        const Raw<TR, true> r = res.get(u);
        F2 w[4];
        w2.get(post_weight, u, w);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v[u][i] = fma2(a1, r.pair(i), q.pair(i) * k1 * w[i]);
          sq = fma2(v[u][i], v[u][i], sq);
        }
        store_unit(row16<TR>(p.res_out, t), m[u], v[u]);
      }
      __syncwarp();
      copy(t + ring * step, slot, next);
      slot = slot + 1 == ring ? 0 : slot + 1;
      const bool more = t + step < p.T;
      s[0] = sum(sq);
      s[1] = 0.0f;
      if (more) {
        ring_wait(ring);
        place(slot);
        next_squares();
      }
      if (more || p.x.p != nullptr) group_sum(g, s);
      if (p.x.p == nullptr) continue;
      const F2 k2 = f2(rsqrtf(s[0] * inv + p.pre.eps));
#pragma unroll
      for (int u = 0; u < NV; ++u) {
        if (beyond(m[u])) continue;
        F2 w[4], x[4];
        w1.get(pre_weight, u, w);
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = v[u][i] * k2 * w[i];
        store_unit(row16<TA>(p.x, t), m[u], x);
      }
    }
  }
  for (; !kPipe && t < p.T; t += step) {
    const float gt = token ? gate_act(p.gate_act, next_gate) : 1.0f;
    next_gate = token_gate(p, t + step);
    ring_wait(ring);
    place(slot);
    Slots after = next;
    if constexpr (MODE == kPre) {
#pragma unroll
      for (int u = 0; u < NV; ++u) {
        if (beyond(m[u])) continue;
        const Raw<TR, true> a = res.get(u);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[u][i] = a.pair(i);
      }
      __syncwarp();
      copy(t + ring * step, slot, next);   // the row is in registers
    } else {
      if constexpr (MODE == kPost) {
#pragma unroll
        for (int u = 0; u < NV; ++u) {
          if (beyond(m[u])) continue;
          const Raw<TA, true> a = y.get(u);
#pragma unroll
          for (int i = 0; i < 4; ++i) v[u][i] = a.pair(i);
        }
      } else {
        after.load(p, t + (ring + 1) * step, g.lane);
#pragma unroll
        for (int u = 0; u < NV; ++u)
#pragma unroll
          for (int i = 0; i < 4; ++i) v[u][i] = zero;
        for (int s = 0; s < slots; ++s) {
          const float w = __shfl_sync(0xFFFFFFFFu, s0.w, s);
          const int r = __shfl_sync(0xFFFFFFFFu, s0.row, s);
          if (r >= 0) {
#pragma unroll
            for (int u = 0; u < NV; ++u) {
              if (beyond(m[u])) continue;
              const Raw<TA, true> a = y.get(u);
#pragma unroll
              for (int i = 0; i < 4; ++i) v[u][i] = fma2(f2(w), a.pair(i), v[u][i]);
            }
          }
          y.at += Act::kPlaces;
        }
        if (p.y_out.p != nullptr) {
#pragma unroll
          for (int u = 0; u < NV; ++u) store_unit(row16<TA>(p.y_out, t), m[u], v[u]);
        }
      }
      float mu = 0.0f, rstd = 1.0f;
      if (PLAIN || p.post.kind != MOE_NORM_NONE) stats(p.post, mu, rstd);
      const float k = full || token ? p.branch_scale * gt : 1.0f;
      const F2 k1 = f2(rstd * k), k0 = f2(-mu * rstd * k), a1 = f2(p.res_scale);
#pragma unroll
      for (int u = 0; u < NV; ++u) {
        if (beyond(m[u])) continue;
        const Raw<TR, true> r = res.get(u);
        F2 w[4];
        w2.get(post_weight, u, w);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          v[u][i] = (PLAIN ? v[u][i] * k1 : fma2(v[u][i], k1, k0)) * w[i];
        if constexpr (BIAS) {
          F2 b[4];
          b2.get(post_bias, u, b);
#pragma unroll
          for (int i = 0; i < 4; ++i) v[u][i] = fma2(b[i], f2(k), v[u][i]);
        }
        if (full) {
          Raw<TA, true> q;
          q.template load<true>(row16<const TA>(p.gate_rows, t), m[u]);
          F2 gv[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) gv[i] = q.pair(i);
          gate_unit(p.gate_act, gv);
#pragma unroll
          for (int i = 0; i < 4; ++i) v[u][i] = v[u][i] * gv[i];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) v[u][i] = fma2(a1, r.pair(i), v[u][i]);
        store_unit(row16<TR>(p.res_out, t), m[u], v[u]);
      }
      __syncwarp();
      copy(t + ring * step, slot, next);
    }
    if (p.x.p != nullptr) {
      float mu, rstd;
      stats(p.pre, mu, rstd);
      const F2 k1 = f2(rstd), k0 = f2(-mu * rstd);
#pragma unroll
      for (int u = 0; u < NV; ++u) {
        if (beyond(m[u])) continue;
        F2 w[4], x[4];
        w1.get(pre_weight, u, w);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          x[i] = (PLAIN ? v[u][i] * k1 : fma2(v[u][i], k1, k0)) * w[i];
        if constexpr (BIAS) {
          F2 b[4];
          b1.get(pre_bias, u, b);
#pragma unroll
          for (int i = 0; i < 4; ++i) x[i] = x[i] + b[i];
        }
        store_unit(row16<TA>(p.x, t), m[u], x);
      }
    }
    slot = slot + 1 == ring ? 0 : slot + 1;
    if constexpr (MODE == kRouted) {
      s0 = ring > 1 ? s1 : next;
      s1 = ring > 2 ? s2 : next;
      s2 = next;
      next = after;
    }
  }
}

// The plain form (PLAIN): RMS norms without biases and no gate tensor, where the
// means and what depends on them drop out of the arithmetic at compile time
// (post norm over an fp32 residual, 16384 x 7168: 286 instead of 303 us).
bool plain_fwd(const BlockArgs& a, bool post) {
  return a.post.b == nullptr && a.pre.b == nullptr &&
         (a.x.p == nullptr || a.pre.kind == MOE_NORM_RMS) &&
         (!post || (a.post.kind == MOE_NORM_RMS && a.gate != MOE_GATE_FULL));
}

// Launches the ring's kernel; `none` set where not one row fits the ring.
template <typename TA, typename TR, int NV, int MODE>
cudaError_t launch_ring(const BlockArgs& a, int sms, bool& none, cudaStream_t s) {
  const int groups = kBlockThreads / a.tpr, threads = groups * a.tpr;
  const int slots = MODE == kRouted ? a.k : MODE == kPost ? 1 : 0;
  const size_t row = static_cast<size_t>(RowPart<TR, NV, true>::kPieces +
                                         slots * RowPart<TA, NV, true>::kPieces) *
                     kBlockThreads * 16;
  int ring = static_cast<int>(kBlockSmem / row);
  none = ring == 0;
  if (none) return cudaSuccess;
  if (ring > kRing) ring = kRing;
  const bool bias = a.post.b != nullptr || a.pre.b != nullptr;
  const bool plain = plain_fwd(a, MODE != kPre);
  auto* k = plain  ? k_block_fwd_ring<TA, TR, NV, MODE, false, true>
            : bias ? k_block_fwd_ring<TA, TR, NV, MODE, true, false>
                   : k_block_fwd_ring<TA, TR, NV, MODE, false, false>;
  static std::atomic<uint64_t> done[3];
  const cudaError_t e = allow_ring(reinterpret_cast<const void*>(k), done[plain ? 0 : bias ? 1 : 2]);
  if (e != cudaSuccess) return e;
  int blocks = (a.T + groups - 1) / groups;
  if (blocks > sms) blocks = sms;
  k<<<blocks, threads, ring * row, s>>>(a, ring);
  return cudaGetLastError();
}

template <typename TA, typename TR, int NV>
cudaError_t launch_ring_mode(const BlockArgs& a, bool post, int sms, bool& none, cudaStream_t s) {
  if (!post) return launch_ring<TA, TR, NV, kPre>(a, sms, none, s);
  if (a.row_of == nullptr) return launch_ring<TA, TR, NV, kPost>(a, sms, none, s);
  return launch_ring<TA, TR, NV, kRouted>(a, sms, none, s);
}

template <typename TA, typename TR, int NV, bool VEC, bool HOIST>
cudaError_t launch_nv(const BlockArgs& a, bool post, cudaStream_t s) {
  // several rows a block where a warp holds one, else one
  const int groups = a.tpr == 32 ? 4 : 1;
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

// Channels an SM up to which the calls are few rows.  Measured, post norm with
// the next norm in bf16, one group a row against the ring: 2048 channels, 608
// tokens 5.6 and 6.8 us, 1216 tokens 8.2 and 7.0; 1024 channels, 608 tokens 3.5
// and 4.5, 1216 tokens 5.5 and 4.7; 4096 channels, 456 tokens 8.2 and 7.0.
constexpr long long kFewChannels = 8192;

template <typename TA, typename TR>
cudaError_t launch_block_fwd_types(BlockArgs a, bool post, int sms, cudaStream_t s) {
  const int units = (a.d + kUnit - 1) / kUnit;
  auto threads = [&](int nv) { return ((units + nv - 1) / nv + 31) / 32 * 32; };
  if (a.vec && static_cast<long long>(a.T) * a.d > kFewChannels * sms) {
    bool none = false;
    // two units a thread where a row has them, and four where their parameters
    // still fit the registers: more groups, whose sums wait apart.  k is not
    // looked at, and four units halve the expert rows that the ring can take: 5
    // a token in bf16, 4 over an fp32 residual, 2 in fp32 (two units: 12, 11, 5).
    // Beyond that the few rows' kernel takes the call: 4096 x 2048, k = 6, 62 us
    // in the plain form without the ring, 41 us in the general one with it
    const bool four = units > 2 * kBlockThreads || (units > 128 && plain_fwd(a, post));
    const int nv = units <= 32 ? 1 : four ? 4 : 2;
    a.tpr = threads(nv);
    const cudaError_t e = nv == 1   ? launch_ring_mode<TA, TR, 1>(a, post, sms, none, s)
                          : nv == 2 ? launch_ring_mode<TA, TR, 2>(a, post, sms, none, s)
                                    : launch_ring_mode<TA, TR, 4>(a, post, sms, none, s);
    if (!none) return e;
  }
  if (a.vec && units <= 2 * kBlockThreads) {
    const bool one = units <= kBlockThreads;
    a.tpr = threads(one ? 1 : 2);
    return one ? launch_nv<TA, TR, 1, true, true>(a, post, s)
               : launch_nv<TA, TR, 2, true, true>(a, post, s);
  }
  const bool wide = units > 2 * kBlockThreads / 2;
  a.tpr = threads(wide ? 8 : 2);
  return wide ? launch_nv<TA, TR, 8, false, false>(a, post, s)
              : launch_nv<TA, TR, 2, false, false>(a, post, s);
}

}  // namespace moe
