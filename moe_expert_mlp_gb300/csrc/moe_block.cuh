// Device functions shared by the forward and backward kernels of the residual
// block's norms (moe_block_fwd.cu, moe_block_bwd.cu): how a row is spread over
// a group of threads, and sums over the group.
//
// A row of d channels belongs to a group of `tpr` threads (a multiple of 32),
// each holding kUnit = 8 channels in each of NV units.  With 16-byte aligned
// rows a unit is 8 neighbouring channels (one 16-byte access in bf16, two in
// fp32); otherwise its channels lie tpr apart, so that the warp's single
// elements are still neighbours.  A block holds several groups when rows are
// short.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "moe_internal.h"
#include "moe_ptx.cuh"

namespace moe {

constexpr int kBlockThreads = 512;   // threads of a block at most
constexpr int kUnit = 8;             // channels of a unit
constexpr int kBlockMaxD = 16384;    // 512 threads x 4 units

// Row tensor: element (t, c) at p[t * ld + c].
struct BlockRows {
  char* p;
  long long ld;
};

struct BlockNorm {
  int kind;          // moe_norm_kind_t
  float eps, off;
  const void* w;     // may be null
  const void* b;     // may be null
};

struct BlockArgs {
  int T, d;
  int tpr, nv;       // threads of a group, units of a thread
  int vec;           // every row 16-byte aligned and d % 8 == 0
  int p32;           // parameters are fp32 (else bf16)
  int gate, gate_act;
  float res_scale, branch_scale, dres_scale;
  BlockNorm pre, post;
  BlockRows gate_rows;
  // forward: res -> res_out, x; y (or the expert rows) -> y_out
  // backward: dres_in, dx, res (the normed residual), y -> dres, dy
  BlockRows res, res_out, x, y, y_out;
  BlockRows dres_in, dx, dres, dy;
  // routed branch
  const int32_t* row_of;
  const float* topk_w;
  int k, capacity;
  int* status;
  // backward
  float* part;       // [blocks][accumulators][d]
  BlockRows dgate;   // token, full
};

// Channels of unit u of thread `lane` of its group.
struct UnitMap {
  int c0, step, n;
};

__device__ __forceinline__ UnitMap unit_map(const BlockArgs& p, int lane, int u) {
  UnitMap m;
  if (p.vec) {
    m.c0 = (u * p.tpr + lane) * kUnit;
    m.step = 1;
    m.n = m.c0 < p.d ? kUnit : 0;
  } else {
    m.c0 = u * kUnit * p.tpr + lane;
    m.step = p.tpr;
    m.n = m.c0 < p.d ? min(kUnit, (p.d - m.c0 + p.tpr - 1) / p.tpr) : 0;
  }
  return m;
}

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}

__device__ __forceinline__ void unpack8(const uint4& w, float (&v)[8]) {
  v[0] = bf16_lo(w.x);
  v[1] = bf16_hi(w.x);
  v[2] = bf16_lo(w.y);
  v[3] = bf16_hi(w.y);
  v[4] = bf16_lo(w.z);
  v[5] = bf16_hi(w.z);
  v[6] = bf16_lo(w.w);
  v[7] = bf16_hi(w.w);
}

// The unit's elements of one row, 0 past the row's end.
template <typename T>
__device__ __forceinline__ void load_unit(const T* row, const UnitMap& m, bool vec, float (&v)[8]) {
  if (vec) {
    if (m.n) {
      if constexpr (sizeof(T) == 2) {
        unpack8(*reinterpret_cast<const uint4*>(row + m.c0), v);
      } else {
        const float4 a = *reinterpret_cast<const float4*>(row + m.c0);
        const float4 b = *reinterpret_cast<const float4*>(row + m.c0 + 4);
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
        v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = 0.0f;
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = e < m.n ? to_f32(row[m.c0 + e * m.step]) : 0.0f;
  }
}

template <typename T>
__device__ __forceinline__ void store_unit(T* row, const UnitMap& m, bool vec, const float (&v)[8]) {
  if (vec) {
    if (m.n) {
      if constexpr (sizeof(T) == 2) {
        *reinterpret_cast<uint4*>(row + m.c0) =
            make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                       pack_bf16x2(v[6], v[7]));
      } else {
        *reinterpret_cast<float4*>(row + m.c0) = make_float4(v[0], v[1], v[2], v[3]);
        *reinterpret_cast<float4*>(row + m.c0 + 4) = make_float4(v[4], v[5], v[6], v[7]);
      }
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < m.n) row[m.c0 + e * m.step] = from_f32<T>(v[e]);
  }
}

// The unit's elements of a parameter vector (bf16 or fp32), `absent` where
// there is none.
__device__ __forceinline__ void load_param(const void* w, const BlockArgs& p, const UnitMap& m,
                                           float off, float absent, float (&v)[8]) {
  if (w == nullptr) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = absent;
    return;
  }
  if (p.p32)
    load_unit(static_cast<const float*>(w), m, p.vec, v);
  else
    load_unit(static_cast<const __nv_bfloat16*>(w), m, p.vec, v);
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] += off;
}

template <typename T>
__device__ __forceinline__ T* row_ptr(const BlockRows& r, int t) {
  return reinterpret_cast<T*>(r.p) + static_cast<long long>(t) * r.ld;
}

// Gate value and the derivative of its activation.
__device__ __forceinline__ float gate_act(int act, float g) {
  if (act == MOE_GATE_ACT_SIGMOID) return 1.0f / (1.0f + expf(-g));
  if (act == MOE_GATE_ACT_TANH) return tanhf(g);
  return g;
}
__device__ __forceinline__ float gate_slope(int act, float v) {
  if (act == MOE_GATE_ACT_SIGMOID) return v * (1.0f - v);
  if (act == MOE_GATE_ACT_TANH) return 1.0f - v * v;
  return 1.0f;
}

// A thread's place: its group's row, its place in the group, and the group's
// shared partials (two sets used in turn: a set is written again only behind
// the other set's barrier, when every thread has read it).
struct Group {
  int lane;      // thread of the group
  int id;        // group of the block
  int warps;     // warps of the group
  float4* red;   // [2][warps]
  int turn;
};

__device__ __forceinline__ Group make_group(const BlockArgs& p, float4* red) {
  Group g;
  g.id = threadIdx.x / p.tpr;
  g.lane = threadIdx.x - g.id * p.tpr;
  g.warps = p.tpr / 32;
  g.red = red + g.id * 2 * g.warps;
  g.turn = 0;
  return g;
}

// Sums over the group, the same value in every thread of it.
template <int N>
__device__ __forceinline__ void group_sum(Group& g, float (&v)[N]) {
  static_assert(N >= 1 && N <= 4, "one float4 of partials");
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xFFFFFFFFu, v[i], o);
  if (g.warps == 1) return;
  float4* set = g.red + g.turn * g.warps;
  g.turn ^= 1;
  if ((g.lane & 31) == 0) {
    float4 w = make_float4(v[0], 0.0f, 0.0f, 0.0f);
    if constexpr (N > 1) w.y = v[1];
    if constexpr (N > 2) w.z = v[2];
    if constexpr (N > 3) w.w = v[3];
    set[g.lane >> 5] = w;
  }
  asm volatile("bar.sync %0, %1;" ::"r"(g.id + 1), "r"(g.warps * 32) : "memory");
  const int l = g.lane & 31;
  const float4 w = l < g.warps ? set[l] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  v[0] = w.x;
  if constexpr (N > 1) v[1] = w.y;
  if constexpr (N > 2) v[2] = w.z;
  if constexpr (N > 3) v[3] = w.w;
  // at most 16 warps
#pragma unroll
  for (int o = 8; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xFFFFFFFFu, v[i], o);
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = __shfl_sync(0xFFFFFFFFu, v[i], 0);
}

// Blocks whose partial sums the backward's workspace has room for.
constexpr int kBlockBwdMaxParts = 304;

struct BlockGrads {
  bool pre, post, bias;                     // sides present; bias sums kept
  void *dpre_w, *dpre_b, *dpost_w, *dpost_b;
  void* dgate;                              // channel gate
  int acc, parts;                           // set by the launcher
};

cudaError_t launch_block_fwd(const BlockArgs& a, int dtype, int res_dtype, bool post,
                             cudaStream_t s);
cudaError_t launch_block_bwd(const BlockArgs& a, BlockGrads o, int dtype, int res_dtype, int sms,
                             cudaStream_t s);

}  // namespace moe
