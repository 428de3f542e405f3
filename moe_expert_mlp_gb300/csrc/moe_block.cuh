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
constexpr int kFewRows = 2;          // rows an SM up to which a row's latency counts

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
  int tpr;           // threads of a group (the launchers')
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

// Channels of unit u of thread `lane` of its group: c0, c0 + step, ..., those
// below d.  VEC: 8 neighbours, all or none.
template <bool VEC>
struct Unit {
  int c0, d, tpr;
  __device__ __forceinline__ Unit() {}
  __device__ __forceinline__ Unit(const BlockArgs& p, int lane, int u) : d(p.d), tpr(p.tpr) {
    c0 = VEC ? (u * p.tpr + lane) * kUnit : u * kUnit * p.tpr + lane;
  }
  __device__ __forceinline__ int at(int e) const { return VEC ? c0 + e : c0 + e * tpr; }
  __device__ __forceinline__ bool has(int e) const { return VEC ? c0 < d : c0 + e * tpr < d; }
};

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

// 16 bytes of a row, read once: they do not displace the parameters in L1.
__device__ __forceinline__ uint4 load16_once(const void* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// A unit's 8 elements as they lie in memory (VEC: 16 bytes in bf16, 32 in
// fp32; else one register each), 0 past the row's end.
template <typename T, bool VEC>
struct Raw {
  static constexpr int kWords = VEC ? 2 * sizeof(T) : 8;
  uint32_t w[kWords];

  template <bool ONCE>
  __device__ __forceinline__ void load(const T* row, const Unit<VEC>& m) {
    if constexpr (VEC) {
#pragma unroll
      for (int i = 0; i < kWords / 4; ++i) {
        uint4 q = make_uint4(0, 0, 0, 0);
        const uint4* from = reinterpret_cast<const uint4*>(row + m.c0) + i;
        if (m.has(0)) q = ONCE ? load16_once(from) : *from;
        w[4 * i] = q.x, w[4 * i + 1] = q.y, w[4 * i + 2] = q.z, w[4 * i + 3] = q.w;
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e] = m.has(e) ? __float_as_uint(to_f32(row[m.at(e)])) : 0u;
    }
  }
  __device__ __forceinline__ float get(int e) const {
    if constexpr (VEC && sizeof(T) == 2)
      return e & 1 ? bf16_hi(w[e / 2]) : bf16_lo(w[e / 2]);
    else
      return __uint_as_float(w[e]);
  }
};

// The unit's elements of one row: read once, past L1.
template <typename T, bool VEC>
__device__ __forceinline__ void load_row(const T* row, const Unit<VEC>& m, float (&v)[8]) {
  Raw<T, VEC> r;
  r.template load<true>(row, m);
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = r.get(e);
}

template <typename T, bool VEC>
__device__ __forceinline__ void store_unit(T* row, const Unit<VEC>& m, const float (&v)[8]) {
  if constexpr (VEC) {
    if (m.has(0)) {
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
      if (m.has(e)) row[m.at(e)] = from_f32<T>(v[e]);
  }
}

// The unit's elements of a parameter vector (bf16 or fp32) plus `off`,
// `absent` where there is none.
template <bool VEC>
__device__ __forceinline__ void load_param(const void* w, const BlockArgs& p, const Unit<VEC>& m,
                                           float off, float absent, float (&v)[8]) {
  if (w == nullptr) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = absent;
  } else if (p.p32) {
    Raw<float, VEC> r;
    r.template load<false>(static_cast<const float*>(w), m);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = r.get(e) + off;
  } else {
    Raw<__nv_bfloat16, VEC> r;
    r.template load<false>(static_cast<const __nv_bfloat16*>(w), m);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = r.get(e) + off;
  }
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

// Forward (POST: the post norm), for one pair of activation and residual types.
template <typename TA, typename TR>
cudaError_t launch_block_fwd_types(BlockArgs a, bool post, int sms, cudaStream_t s);
// Backward over the rows; sets o.parts.
template <typename TA, typename TR>
cudaError_t launch_block_bwd_types(BlockArgs a, BlockGrads& o, int sms, cudaStream_t s);
cudaError_t launch_block_bwd(const BlockArgs& a, BlockGrads o, int dtype, int res_dtype, int sms,
                             cudaStream_t s);

}  // namespace moe
