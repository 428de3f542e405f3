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
// memory (cp.async), and waits for no one else's (an fp32 warp: for its own
// threads').  Measured: pre norm, 16384 x 4096 in bf16, 84 us = 6.4 TB/s, 94 % of
// the rate of a copy; both norms, 16384 x 7168, 246 us = 5.7 TB/s (84 %), where
// one group of 14 warps has the SM, about 700 instructions a row and warp (two
// sums a row instead of one that meets the next row's took 270 us; 28 warps of
// one unit a thread 339 us, as the sums wait for all of them; four units a
// thread do not fit the registers);
// post norm with a token gate, 4096 x 2048, 17 us = 3.0 TB/s, a fifth of it
// the launch of the sums over blocks; its 27 rows an SM go through four groups,
// whose rows wait for their sums one after another (meeting the next row's, as
// with both norms, was not tried there).  The general form, whose three sums a
// row follow each other: pre layer norm with bias, 16384 x 4096, 123 us = 4.4 TB/s;
// both layer norms, 16384 x 7168, 370 us = 3.8 TB/s, with biases 695 us (their
// sums take the weights' registers, which come from L1 then), with a gate tensor
// 800 us.  Rows that are not aligned are read element by
// element into registers, with the next row called into L2: 1001 x 1441 in fp32,
// two layer norms and a gate tensor, 36 us = 1.3 TB/s.
#pragma once

#include "moe_block.cuh"

namespace moe {
namespace {

// Pieces of a ring row: the tensors that the kernel copies.
template <typename TA, typename TR, int NV, bool VEC, bool PRE, bool POST>
__host__ __device__ constexpr int ring_pieces() {
  return RowPart<TR, NV, VEC>::kPieces * (PRE ? 2 : 1) +
         RowPart<TA, NV, VEC>::kPieces * ((PRE ? 1 : 0) + (POST ? 1 : 0));
}

template <typename TA, typename TR, int NV, bool VEC, bool PRE, bool POST, bool BIAS, bool PLAIN>
__global__ void __launch_bounds__(kBlockThreads, 1)
    k_block_bwd(const __grid_constant__ BlockArgs p, int ring) {
  constexpr int kSides = (PRE ? 1 : 0) + (POST ? 1 : 0);
  constexpr int kAcc = kSides * (BIAS ? 2 : 1);
  constexpr int kS1 = PRE ? (BIAS ? 2 : 1) : 0;        // the post norm's first sum
  constexpr bool kHeld = NV == 1 || (NV == 2 && !BIAS);
  constexpr int kPieces = ring_pieces<TA, TR, NV, VEC, PRE, POST>();
  constexpr bool kPipe = PLAIN && PRE && POST && kPieces * kBlockThreads * 16 * 2 <= kBlockSmem;
  __shared__ float red[kRedFloats];
  extern __shared__ uint4 dyn[];                 // the ring; then the groups' sums
  Group<true> g = make_group<true>(p, red);
  const int groups = blockDim.x / p.tpr;
  const float inv = 1.0f / static_cast<float>(p.d);
  const bool pre_layer = !PLAIN && PRE && p.pre.kind == MOE_NORM_LAYER;
  const bool normed = POST && (PLAIN || p.post.kind != MOE_NORM_NONE);
  const bool post_layer = !PLAIN && POST && p.post.kind == MOE_NORM_LAYER;
  const bool full = !PLAIN && p.gate == MOE_GATE_FULL, token = p.gate == MOE_GATE_TOKEN;
  Unit<VEC> m[NV];
#pragma unroll
  for (int u = 0; u < NV; ++u) m[u] = Unit<VEC>(p, g.lane, u);

  // the ring's places of this thread, and the copy of row t into slot i
  RowPart<TR, NV, VEC> dres_in, res;
  RowPart<TA, NV, VEC> dx, y;
  auto place = [&](int slot) {
    if constexpr (VEC) {
      uint4* at = dyn + slot * kPieces * kBlockThreads;
      dres_in.at = at;
      at += RowPart<TR, NV, VEC>::kPlaces;
      if constexpr (PRE) {
        res.at = at;
        at += RowPart<TR, NV, VEC>::kPlaces;
        dx.at = at;
        at += RowPart<TA, NV, VEC>::kPlaces;
      }
      y.at = at;
    }
  };
  auto copy = [&](int t, int slot) {
    if constexpr (VEC) {
      if (t < p.T) {
        place(slot);
        if constexpr (PRE) {
          res.copy(row_at<VEC, const TR>(p.res, t), m);
          dx.copy(row_at<VEC, const TA>(p.dx, t), m);
        }
        if constexpr (POST) y.copy(row_at<VEC, const TA>(p.y, t), m);
        if (p.dres_in.p != nullptr) dres_in.copy(row_at<VEC, const TR>(p.dres_in, t), m);
      }
      copies_commit();   // one group a row, empty past the end
    }
  };

  const int step = gridDim.x * groups;
  int t = blockIdx.x * groups + g.id;
  for (int i = 0; i < ring; ++i) copy(t + i * step, i);

  // the pre norm's weights, and the post norm's times gate and scale where
  // neither changes from token to token
  auto pre_weight = [&](int u, F2 (&v)[4]) { load_param(p.pre.w, p, m[u], p.pre.off, 1.0f, v); };
  auto post_weight = [&](int u, F2 (&v)[4]) {
    load_param(p.post.w, p, m[u], p.post.off, 1.0f, v);
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
  Weights<NV, kHeld> w1, w2;
  if constexpr (PRE) w1.fetch(pre_weight);
  if constexpr (POST) w2.fetch(post_weight);

  F2 acc[kAcc][NV][4];
#pragma unroll
  for (int a = 0; a < kAcc; ++a)
#pragma unroll
    for (int u = 0; u < NV; ++u)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[a][u][i] = f2(0.0f);

  if constexpr (kPipe) {
    // Both sides in the plain form: this row's sum over the post norm and the
    // next row's three sums meet in one, so that a row waits once.
    float s[4];                                  // post norm's; squares, dxh v, y's squares
    auto next_sums = [&]() {
      F2 s1 = f2(0.0f), s2 = s1, s3 = s1;
#pragma unroll
      for (int u = 0; u < NV; ++u) {
        if (beyond(m[u])) continue;
        const Raw<TR, VEC> a = res.get(u);
        const Raw<TA, VEC> b = dx.get(u), c = y.get(u);
        F2 w[4];
        w1.get(pre_weight, u, w);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const F2 v = a.pair(i), q = c.pair(i);
          s1 = fma2(v, v, s1);
          s2 = fma2(b.pair(i) * w[i], v, s2);
          s3 = fma2(q, q, s3);
        }
      }
      s[1] = sum(s1), s[2] = sum(s2), s[3] = sum(s3);
    };
    float next_gate = token_gate(p, t);
    int slot = 0;
    if (t < p.T) {
      ring_wait(ring);
      place(0);
      next_sums();
      s[0] = 0.0f;
      group_sum(g, s);
    }
    for (; t < p.T; t += step) {
      const float rstd = rsqrtf(s[1] * inv + p.pre.eps);
      const float rstd2 = rsqrtf(s[3] * inv + p.post.eps);
      const float k1 = -(rstd * (s[2] * inv * rstd)) * rstd;
      const float gt = token ? gate_act(p.gate_act, next_gate) : 1.0f;
      next_gate = token_gate(p, t + step);
      place(slot);
      F2 D[NV][4], e = f2(0.0f);
      const F2 r2 = f2(rstd), kk1 = f2(k1);
#pragma unroll
      for (int u = 0; u < NV; ++u) {
        if (beyond(m[u])) continue;
        if (p.dres_in.p != nullptr) {
          const Raw<TR, VEC> q = dres_in.get(u);
#pragma unroll
          for (int i = 0; i < 4; ++i) D[u][i] = f2(p.dres_scale) * q.pair(i);
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) D[u][i] = f2(0.0f);
        }
        const Raw<TR, VEC> a = res.get(u);
        const Raw<TA, VEC> b = dx.get(u), c = y.get(u);
        F2 w[4], ww[4];
        w1.get(pre_weight, u, w);
        w2.get(post_weight, u, ww);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const F2 v = a.pair(i), d = b.pair(i);
          acc[0][u][i] = fma2(d, v * r2, acc[0][u][i]);
          D[u][i] = fma2(d * w[i], r2, fma2(v, kk1, D[u][i]));
          e = fma2(D[u][i] * ww[i], c.pair(i), e);
        }
        if (p.dres.p != nullptr) store_unit(row_at<VEC, TR>(p.dres, t), m[u], D[u]);
      }
      s[0] = sum(e);
      s[1] = s[2] = s[3] = 0.0f;
      const int behind = slot + 1 == ring ? 0 : slot + 1;
      if (t + step < p.T) {
        ring_wait(ring - 1);
        slot = behind;
        place(slot);
        next_sums();
        slot = behind == 0 ? ring - 1 : behind - 1;
      }
      group_sum(g, s);
      const float e2 = s[0];
      if (token && p.dgate.p != nullptr && g.lane == 0)
        *row_ptr<float>(p.dgate, t) = p.branch_scale * rstd2 * e2 * gate_slope(p.gate_act, gt);
      const float scale = token ? p.branch_scale * gt : 1.0f;
      const F2 kk2 = f2(rstd2 * scale), ky = f2(-(rstd2 * (scale * e2 * inv * rstd2)) * rstd2);
      const F2 rg = f2(rstd2 * gt);              // xhat, with the token's gate
      place(slot);
#pragma unroll
      for (int u = 0; u < NV; ++u) {
        if (beyond(m[u])) continue;
        const Raw<TA, VEC> c = y.get(u);
        F2 w[4], dy[4];
        w2.get(post_weight, u, w);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const F2 v = c.pair(i);
          acc[kS1][u][i] = fma2(D[u][i], v * rg, acc[kS1][u][i]);
          dy[i] = fma2(D[u][i] * w[i], kk2, v * ky);
        }
        store_unit(row_at<VEC, TA>(p.dy, t), m[u], dy);
      }
      __syncwarp();
      copy(t + ring * step, slot);
      slot = behind;
    }
  }

  // v - mu of the row's elements
  auto centred = [](F2 v, float mu) { return PLAIN ? v : v + f2(-mu); };
  float next_gate = token_gate(p, t);
  int slot = 0;
  for (; !kPipe && t < p.T; t += step) {
    if constexpr (VEC) {
      ring_wait(ring);
      place(slot);
    } else {
      if constexpr (PRE) {
        res.fetch(row_at<VEC, const TR>(p.res, t), m);
        dx.fetch(row_at<VEC, const TA>(p.dx, t), m);
      }
      if constexpr (POST) y.fetch(row_at<VEC, const TA>(p.y, t), m);
      if (p.dres_in.p != nullptr) dres_in.fetch(row_at<VEC, const TR>(p.dres_in, t), m);
      // the next row into L2, a line a thread
      if (t + step < p.T) {
        const int at = g.lane * 128;
        auto line = [&](const BlockRows& r, int size) {
          if (r.p != nullptr && at < p.d * size)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(r.p + (t + step) * r.ld * size + at));
        };
        if constexpr (PRE) {
          line(p.res, sizeof(TR));
          line(p.dx, sizeof(TA));
        }
        if constexpr (POST) line(p.y, sizeof(TA));
        line(p.dres_in, sizeof(TR));
        if (full) line(p.gate_rows, sizeof(TA));
      }
    }
    const float gt = token ? gate_act(p.gate_act, next_gate) : 1.0f;
    next_gate = token_gate(p, t + step);
    float mu1 = 0.0f, mu2 = 0.0f;
    if (pre_layer || post_layer) {
      F2 a1 = f2(0.0f), a2 = f2(0.0f);
#pragma unroll
      for (int u = 0; u < NV; ++u) {
        if (beyond(m[u])) continue;
        if constexpr (PRE) {
          const Raw<TR, VEC> a = res.get(u);
#pragma unroll
          for (int i = 0; i < 4; ++i) a1 = a1 + a.pair(i);
        }
        if constexpr (POST) {
          const Raw<TA, VEC> a = y.get(u);
#pragma unroll
          for (int i = 0; i < 4; ++i) a2 = a2 + a.pair(i);
        }
      }
      float s[2] = {sum(a1), sum(a2)};
      group_sum(g, s);
      if (pre_layer) mu1 = s[0] * inv;
      if (post_layer) mu2 = s[1] * inv;
    }

    // Sums over the row.  With a pre norm: its squares, dxh, dxh (r' - mu) and
    // the post norm's squares; without: the post norm's own, as D is known.
    F2 D[NV][4];
    const F2 zero = f2(0.0f);
    auto load_D = [&](int u, F2 (&d)[4]) {
      if (p.dres_in.p != nullptr) {
        const Raw<TR, VEC> a = dres_in.get(u);
#pragma unroll
        for (int i = 0; i < 4; ++i) d[i] = f2(p.dres_scale) * a.pair(i);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) d[i] = zero;
      }
    };
    // The post norm's sums: dxh, dxh (y - mu), D bias.  The token's gate, and
    // the scale with a token or full gate, the caller applies to the sums.
    // D is 0 past the row's end.
    auto post_sums = [&](int u, F2& s1, F2& s2, F2& s3) {
      const Raw<TA, VEC> a = y.get(u);
      F2 w[4];
      w2.get(post_weight, u, w);
      if (full) {
        Raw<TA, VEC> r;
        r.template load<true>(row_at<VEC, const TA>(p.gate_rows, t), m[u]);
        F2 q[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) q[i] = r.pair(i);
        gate_unit(p.gate_act, q);
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = w[i] * q[i];
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const F2 dxh = D[u][i] * w[i];
        if (!PLAIN) s1 = s1 + dxh;
        s2 = fma2(dxh, centred(a.pair(i), mu2), s2);
      }
      if (!PLAIN && token && p.post.b != nullptr) {
        F2 b[4];
        load_param(p.post.b, p, m[u], 0.0f, 0.0f, b);
#pragma unroll
        for (int i = 0; i < 4; ++i) s3 = fma2(D[u][i], b[i], s3);
      }
    };
    auto post_squares = [&](int u, F2& q) {
      const Raw<TA, VEC> a = y.get(u);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const F2 c = within(m[u], i, centred(a.pair(i), mu2));
        q = fma2(c, c, q);
      }
    };
    float rstd2 = 1.0f;
    if constexpr (PRE) {
      F2 s0 = zero, s1 = zero, s2 = zero, s3 = zero;
#pragma unroll
      for (int u = 0; u < NV; ++u) {
        if (beyond(m[u])) continue;
        const Raw<TR, VEC> a = res.get(u);
        const Raw<TA, VEC> b = dx.get(u);
        F2 w[4];
        w1.get(pre_weight, u, w);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const F2 c = within(m[u], i, centred(a.pair(i), mu1));
          const F2 dxh = b.pair(i) * w[i];
          s0 = fma2(c, c, s0);
          if (!PLAIN) s1 = s1 + dxh;
          s2 = fma2(dxh, c, s2);
        }
        if (normed) post_squares(u, s3);
      }
      float s[4] = {sum(s0), sum(s1), sum(s2), sum(s3)};
      if constexpr (PLAIN && !POST) {
        float q[2] = {s[0], s[2]};
        group_sum(g, q);
        s[0] = q[0], s[2] = q[1];
      } else {
        group_sum(g, s);
      }
      const float rstd = rsqrtf(s[0] * inv + p.pre.eps);
      if (normed) rstd2 = rsqrtf(s[3] * inv + p.post.eps);
      // rstd (dxh - m0 - xhat m1) = rstd dxh + k1 r' + k0
      const float m1 = s[2] * inv * rstd, k1 = -(rstd * m1) * rstd;
      const float k0 = (pre_layer ? -rstd * (s[1] * inv) : 0.0f) - k1 * mu1;
      const F2 r2 = f2(rstd), c2 = f2(-mu1 * rstd), kk1 = f2(k1), kk0 = f2(k0);
#pragma unroll
      for (int u = 0; u < NV; ++u) {
        if (beyond(m[u])) continue;
        load_D(u, D[u]);
        const Raw<TR, VEC> a = res.get(u);
        const Raw<TA, VEC> b = dx.get(u);
        F2 w[4];
        w1.get(pre_weight, u, w);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const F2 v = a.pair(i), d = b.pair(i);
          acc[0][u][i] = fma2(d, PLAIN ? v * r2 : fma2(v, r2, c2), acc[0][u][i]);
          if constexpr (BIAS) acc[1][u][i] = acc[1][u][i] + d;     // dx is 0 past the end
          const F2 join = PLAIN ? fma2(v, kk1, D[u][i]) : fma2(v, kk1, D[u][i] + kk0);
          D[u][i] = within(m[u], i, fma2(d * w[i], r2, join));
        }
        if (p.dres.p != nullptr) store_unit(row_at<VEC, TR>(p.dres, t), m[u], D[u]);
      }
    } else {
#pragma unroll
      for (int u = 0; u < NV; ++u) {
        if (beyond(m[u])) continue;
        load_D(u, D[u]);
        if (p.dres.p != nullptr) store_unit(row_at<VEC, TR>(p.dres, t), m[u], D[u]);
      }
    }

    if constexpr (POST) {
      F2 s1 = zero, s2 = zero, s3 = zero;
      float e1 = 0.0f, e2 = 0.0f, e3 = 0.0f;
      if (normed || token) {
        F2 s0 = zero;
#pragma unroll
        for (int u = 0; u < NV; ++u) {
          if (beyond(m[u])) continue;
          post_sums(u, s1, s2, s3);
          if (!PRE && normed) post_squares(u, s0);
        }
        if constexpr (PRE) {
          if constexpr (PLAIN) {
            float s[1] = {sum(s2)};
            group_sum(g, s);
            e2 = s[0];
          } else {
            float s[3] = {sum(s1), sum(s2), sum(s3)};
            group_sum(g, s);
            e1 = s[0], e2 = s[1], e3 = s[2];
          }
        } else if constexpr (PLAIN) {
          float s[2] = {sum(s2), sum(s0)};
          group_sum(g, s);
          e2 = s[0];
          rstd2 = rsqrtf(s[1] * inv + p.post.eps);
        } else {
          float s[4] = {sum(s1), sum(s2), sum(s3), sum(s0)};
          group_sum(g, s);
          e1 = s[0], e2 = s[1], e3 = s[2];
          if (normed) rstd2 = rsqrtf(s[3] * inv + p.post.eps);
        }
      }
      if (token && p.dgate.p != nullptr && g.lane == 0)
        *row_ptr<float>(p.dgate, t) =
            p.branch_scale * (rstd2 * e2 + e3) * gate_slope(p.gate_act, gt);
      // dy = rstd (scale D w - m0 - xhat m1) = k2 D w + k1 y + k0
      const float scale = token ? p.branch_scale * gt : full ? p.branch_scale : 1.0f;
      const float k2 = normed ? rstd2 * scale : scale;
      const float m1 = scale * e2 * inv * rstd2, k1 = normed ? -(rstd2 * m1) * rstd2 : 0.0f;
      const float k0 = (post_layer ? -rstd2 * (scale * e1 * inv) : 0.0f) - k1 * mu2;
      const F2 r2 = f2(rstd2 * gt), c2 = f2(-mu2 * rstd2 * gt);   // xhat, with the token's gate
      const F2 kk2 = f2(k2), kk1 = f2(k1), kk0 = f2(k0);
#pragma unroll
      for (int u = 0; u < NV; ++u) {
        if (beyond(m[u])) continue;
        const Raw<TA, VEC> a = y.get(u);
        F2 w[4], dy[4];
        w2.get(post_weight, u, w);
        if (full) {
          Raw<TA, VEC> r;
          r.template load<true>(row_at<VEC, const TA>(p.gate_rows, t), m[u]);
          F2 b[4], dg[4];
          load_param(p.post.b, p, m[u], 0.0f, 0.0f, b);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const F2 n = fma2(fma2(a.pair(i), r2, c2), w[i], b[i]);
            const float2 q = parts(r.pair(i));
            const float g0 = gate_act(p.gate_act, q.x), g1 = gate_act(p.gate_act, q.y);
            dg[i] = f2(p.branch_scale) * D[u][i] * n *
                    f2(gate_slope(p.gate_act, g0), gate_slope(p.gate_act, g1));
            D[u][i] = D[u][i] * f2(g0, g1);      // the gate joins the sums
          }
          if (p.dgate.p != nullptr) store_unit(row_at<VEC, TA>(p.dgate, t), m[u], dg);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const F2 v = a.pair(i);                // D is 0 past the row's end
          acc[kS1][u][i] = fma2(D[u][i], PLAIN ? v * r2 : fma2(v, r2, c2), acc[kS1][u][i]);
          if constexpr (BIAS) acc[kS1 + 1][u][i] = fma2(D[u][i], f2(gt), acc[kS1 + 1][u][i]);
        }
        if (normed) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const F2 v = a.pair(i);
            dy[i] = fma2(D[u][i] * w[i], kk2, PLAIN ? v * kk1 : fma2(v, kk1, kk0));
          }
        } else {   // y has no part in dy, not even 0 times an Inf
#pragma unroll
          for (int i = 0; i < 4; ++i) dy[i] = D[u][i] * w[i] * kk2;
        }
        store_unit(row_at<VEC, TA>(p.dy, t), m[u], dy);
      }
    }
    __syncwarp();
    copy(t + ring * step, slot);
    slot = slot + 1 == ring ? 0 : slot + 1;
  }

  // the block's sums: each group's into shared memory where there are several,
  // then channel by channel in the order of the groups
  if constexpr (VEC) copies_wait<0>();
  float* part = p.part + static_cast<long long>(blockIdx.x) * kAcc * p.d;
  auto put = [&](float* to) {
#pragma unroll
    for (int a = 0; a < kAcc; ++a)
#pragma unroll
      for (int u = 0; u < NV; ++u) {
        float v[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 q = parts(acc[a][u][i]);
          v[2 * i] = q.x, v[2 * i + 1] = q.y;
        }
        if constexpr (VEC) {
          if (m[u].has(0)) {
            float4* at = reinterpret_cast<float4*>(to + a * p.d + m[u].c0);
            at[0] = make_float4(v[0], v[1], v[2], v[3]);
            at[1] = make_float4(v[4], v[5], v[6], v[7]);
          }
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (m[u].has(e)) to[a * p.d + m[u].at(e)] = v[e];
        }
      }
  };
  if (groups == 1) {
    put(part);
    return;
  }
  float* sums = reinterpret_cast<float*>(dyn);   // [groups][kAcc][d]
  const int n = kAcc * p.d;
  __syncthreads();                               // the ring is read no more
  put(sums + g.id * n);
  __syncthreads();
  for (int c = threadIdx.x; c < n; c += blockDim.x) {
    float v = 0.0f;
    for (int i = 0; i < groups; ++i) v += sums[i * n + c];
    part[c] = v;
  }
}

template <typename TA, typename TR, int NV, bool VEC, bool PRE, bool POST, bool BIAS, bool PLAIN>
cudaError_t launch_kernel(const BlockArgs& a, int blocks, int groups, cudaStream_t s) {
  constexpr int kAcc = ((PRE ? 1 : 0) + (POST ? 1 : 0)) * (BIAS ? 2 : 1);
  constexpr size_t kRow = static_cast<size_t>(ring_pieces<TA, TR, NV, VEC, PRE, POST>()) *
                          kBlockThreads * 16;
  if constexpr (VEC && kRow > kBlockSmem) {
    // the widest fp32 rows: not one fits the ring
    return launch_kernel<TA, TR, NV, false, PRE, POST, BIAS, false>(a, blocks, groups, s);
  } else {
    constexpr int kFit = kRow == 0 ? 0 : static_cast<int>(kBlockSmem / (kRow == 0 ? 1 : kRow));
    constexpr int ring = kFit > kRing ? kRing : kFit;
    size_t smem = ring * kRow;
    if (groups > 1) {
      const size_t join = static_cast<size_t>(groups) * kAcc * a.d * sizeof(float);
      if (join > smem) smem = join;
    }
    auto* k = k_block_bwd<TA, TR, NV, VEC, PRE, POST, BIAS, PLAIN>;
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = allow_ring(reinterpret_cast<const void*>(k), done);
    if (e != cudaSuccess) return e;
    k<<<blocks, groups * a.tpr, smem, s>>>(a, ring);
    return cudaGetLastError();
  }
}

template <typename TA, typename TR, int NV, bool VEC, bool PRE, bool POST>
cudaError_t launch_sides(const BlockArgs& a, const BlockGrads& o, int groups, cudaStream_t s) {
  if constexpr (VEC && NV <= 2) {
    // the plain form: the means and what depends on them drop out at compile time
    // (both norms, 16384 x 7168: 272 instead of 383 us)
    const bool plain = !o.bias && (!PRE || a.pre.kind == MOE_NORM_RMS) &&
                       (!POST || (a.post.kind == MOE_NORM_RMS && a.post.b == nullptr &&
                                  a.gate != MOE_GATE_FULL));
    if (plain) return launch_kernel<TA, TR, NV, true, PRE, POST, false, true>(a, o.parts, groups, s);
  }
  return o.bias ? launch_kernel<TA, TR, NV, VEC, PRE, POST, true, false>(a, o.parts, groups, s)
                : launch_kernel<TA, TR, NV, VEC, PRE, POST, false, false>(a, o.parts, groups, s);
}

template <typename TA, typename TR, int NV, bool VEC>
cudaError_t launch_nv(const BlockArgs& a, const BlockGrads& o, int groups, cudaStream_t s) {
  if (o.pre && o.post) return launch_sides<TA, TR, NV, VEC, true, true>(a, o, groups, s);
  if (o.pre) return launch_sides<TA, TR, NV, VEC, true, false>(a, o, groups, s);
  return launch_sides<TA, TR, NV, VEC, false, true>(a, o, groups, s);
}

}  // namespace

template <typename TA, typename TR>
cudaError_t launch_block_bwd_types(BlockArgs a, BlockGrads& o, int sms, cudaStream_t s) {
  // two units a thread where a row has them: more groups, whose sums wait apart
  const int units = (a.d + kUnit - 1) / kUnit;
  const int nv = units <= 32 || (!a.vec && units <= kBlockThreads) ? 1
                 : units <= 2 * kBlockThreads                      ? 2
                                                                   : 4;
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
