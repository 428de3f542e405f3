// Device functions shared by the forward and backward kernels of the residual
// block's norms (moe_block_fwd.cuh, moe_block_bwd.cuh): how a row is spread over
// a group of threads, and sums over the group.
//
// A row of d channels belongs to a group of `tpr` threads (a multiple of 32),
// each holding kUnit = 8 channels in each of NV units.  With rows aligned to a
// unit (16 bytes in bf16, 32 in fp32) a unit is 8 neighbouring channels;
// otherwise its channels lie tpr apart, so that the warp's single elements are
// still neighbours.  A block holds several groups when rows are short.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "moe_f2.cuh"
#include "moe_internal.h"
#include "moe_ptx.cuh"

namespace moe {

constexpr int kBlockThreads = 512;   // threads of a block at most
constexpr int kUnit = 8;             // channels of a unit
constexpr int kBlockMaxD = 16384;    // 512 threads x 4 units
constexpr int kBlockMaxT = 1 << 30;    // a few steps of the grid past it stay in 32 bits

// Row tensor: element (t, c) at p[t * ld + c]; ld16: ld in 16-byte steps (rows
// of an aligned call).
struct BlockRows {
  char* p;
  long long ld;
  uint32_t ld16;
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
  int vec;           // every row aligned to a unit, and d % 8 == 0
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
    if constexpr (VEC && ONCE && sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = 0u;
      if (m.has(0)) load32_once(row + m.c0, w);
    } else if constexpr (VEC) {
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
  // elements 2i, 2i + 1
  __device__ __forceinline__ F2 pair(int i) const {
    if constexpr (VEC && sizeof(T) == 2)
      return f2(bf16_lo(w[i]), bf16_hi(w[i]));
    else
      return f2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
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
        store32(row + m.c0, v);
      }
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (m.has(e)) row[m.at(e)] = from_f32<T>(v[e]);
  }
}

template <typename T, bool VEC>
__device__ __forceinline__ void store_unit(T* row, const Unit<VEC>& m, const F2 (&v)[4]) {
  float q[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 a = parts(v[i]);
    q[2 * i] = a.x, q[2 * i + 1] = a.y;
  }
  store_unit(row, m, q);
}

// v where the row has the elements, 0 past its end (VEC: units are skipped as
// a whole there).
template <bool VEC>
__device__ __forceinline__ F2 within(const Unit<VEC>& m, int i, F2 v) {
  if constexpr (VEC) return v;
  const float2 a = parts(v);
  return f2(m.has(2 * i) ? a.x : 0.0f, m.has(2 * i + 1) ? a.y : 0.0f);
}
template <bool VEC>
__device__ __forceinline__ bool beyond(const Unit<VEC>& m) { return VEC && !m.has(0); }

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

template <bool VEC>
__device__ __forceinline__ void load_param(const void* w, const BlockArgs& p, const Unit<VEC>& m,
                                           float off, float absent, F2 (&v)[4]) {
  float q[8];
  load_param(w, p, m, off, absent, q);
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = f2(q[2 * i], q[2 * i + 1]);
}

template <typename T>
__device__ __forceinline__ T* row_ptr(const BlockRows& r, int t) {
  return reinterpret_cast<T*>(r.p) + static_cast<long long>(t) * r.ld;
}

// A row of an aligned call: one wide multiplication.
template <typename T>
__device__ __forceinline__ T* row16(const BlockRows& r, int t) {
  return reinterpret_cast<T*>(r.p + ((static_cast<uint64_t>(static_cast<uint32_t>(t)) * r.ld16) << 4));
}
template <bool VEC, typename T>
__device__ __forceinline__ T* row_at(const BlockRows& r, int t) {
  if constexpr (VEC) return row16<T>(r, t);
  return row_ptr<T>(r, t);
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

// Applies the gate's activation to a unit, leaving the gate's value.
__device__ __forceinline__ void gate_unit(int act, F2 (&v)[4]) {
  if (act == MOE_GATE_ACT_NONE) return;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 a = parts(v[i]);
    v[i] = f2(gate_act(act, a.x), gate_act(act, a.y));
  }
}

// A thread's place: its group's row, its place in the group, and the group's
// shared partials (two sets used in turn: a set is written again only behind
// the other set's barrier, when every thread has read it).  NAMED: a block
// holds several groups of more than a warp, each with its own barrier; a
// kernel with barriers chosen at run time reserves all sixteen, and four such
// blocks fill an SM, so a kernel that shares its SM goes without.
template <bool NAMED>
struct Group {
  int lane;      // thread of the group
  int id;        // group of the block
  int warps;     // warps of the group, at most 16
  float* red;    // [2][warps][4]
  int turn;
};

constexpr int kRedFloats = 2 * kBlockThreads / 32 * 4;

template <bool NAMED>
__device__ __forceinline__ Group<NAMED> make_group(const BlockArgs& p, float* red) {
  Group<NAMED> g;
  g.id = threadIdx.x / p.tpr;
  g.lane = threadIdx.x - g.id * p.tpr;
  g.warps = p.tpr / 32;
  g.red = red + g.id * 2 * g.warps * 4;
  g.turn = 0;
  return g;
}

// Sums over the group, the same bits in every thread of it.  With 2 (or 3, 4)
// values the warp's halves (quarters) take one value each as they fold, so
// that the shuffles are 5 (6) instead of 10 (20); the lanes of a half (quarter)
// then add the warps' partials of its value.
template <int N, bool NAMED>
__device__ __forceinline__ void group_sum(Group<NAMED>& g, float (&v)[N]) {
  static_assert(N >= 1 && N <= 4, "four partials a warp");
  constexpr unsigned kAll = 0xFFFFFFFFu;
  constexpr int kParts = N == 1 ? 1 : N == 2 ? 2 : 4;   // values side by side in a warp
  constexpr int kWide = 32 / kParts;                    // lanes of a value
  const int l = g.lane & 31;
  float a;
  if constexpr (N == 1) {
    a = v[0];
  } else {
    float x = v[0], y = v[1];
    if constexpr (N > 2) {
      const bool up = l & 16;
      const float z = N > 3 ? v[N - 1] : 0.0f;
      x = (up ? v[2] : v[0]) + __shfl_xor_sync(kAll, up ? v[0] : v[2], 16);
      y = (up ? z : v[1]) + __shfl_xor_sync(kAll, up ? v[1] : z, 16);
    }
    const bool up = l & kWide;
    a = (up ? y : x) + __shfl_xor_sync(kAll, up ? x : y, kWide);
  }
#pragma unroll
  for (int o = kWide / 2; o > 0; o >>= 1) a += __shfl_xor_sync(kAll, a, o);
  if (g.warps > 1) {
    float* set = g.red + g.turn * g.warps * 4;
    g.turn ^= 1;
    const int value = l / kWide, at = l % kWide;
    if (at == 0) set[(g.lane >> 5) * 4 + value] = a;
    if constexpr (NAMED)
      asm volatile("bar.sync %0, %1;" ::"r"(g.id + 1), "r"(g.warps * 32) : "memory");
    else
      __syncthreads();
    a = at < g.warps ? set[at * 4 + value] : 0.0f;
    if constexpr (kWide == 8) {
      if (at + 8 < g.warps) a += set[(at + 8) * 4 + value];
    }
#pragma unroll
    for (int o = kWide < 16 ? kWide / 2 : 8; o > 0; o >>= 1) a += __shfl_xor_sync(kAll, a, o);
  }
  if constexpr (N == 1) {
    v[0] = __shfl_sync(kAll, a, 0);   // lanes 16.. hold no warp's partial
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = __shfl_sync(kAll, a, i * kWide);
  }
}

__device__ __forceinline__ void copy16_async(uint32_t to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void copies_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// One row tensor of a row: a thread's units, in the ring (VEC) or in registers.
// In the ring a unit of the block takes kBlockThreads places of 16 bytes (bf16:
// each thread's own) or twice as many (fp32: a warp's 64 in the order of the
// row, so that its copies move whole sectors; every second eight of them are
// swapped in pairs, which keeps the threads' reads off each other's banks).
template <typename T, int NV, bool VEC>
struct RowPart {
  static constexpr int kHalves = sizeof(T) / 2;
  static constexpr int kPieces = VEC ? NV * kHalves : 0;   // kBlockThreads places each
  static constexpr int kUnitBytes = kHalves * kBlockThreads * 16;
  static constexpr int kPlaces = kPieces * kBlockThreads;
  Raw<T, VEC> held[VEC ? 1 : NV];
  uint4* at;     // its places in shared memory

  __device__ __forceinline__ void copy(const T* row, const Unit<VEC> (&m)[NV]) {
    if constexpr (VEC) {
      const int l = threadIdx.x & 31;
      const uint32_t base = smem_u32(at);
#pragma unroll
      for (int u = 0; u < NV; ++u) {
        if constexpr (kHalves == 1) {
          if (m[u].has(0)) copy16_async(base + u * kUnitBytes + threadIdx.x * 16, row + m[u].c0);
        } else {
          const uint32_t to = base + u * kUnitBytes + (threadIdx.x - l) * 32;
          const int c = m[u].c0 - l * kUnit;               // the warp's first channel
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int q = h * 32 + l;
            if (c + q * 4 < m[u].d) copy16_async(to + (q ^ ((q >> 3) & 1)) * 16, row + c + q * 4);
          }
        }
      }
    }
  }
  __device__ __forceinline__ void fetch(const T* row, const Unit<VEC> (&m)[NV]) {
    if constexpr (!VEC) {
#pragma unroll
      for (int u = 0; u < NV; ++u) held[u].template load<true>(row, m[u]);
    }
  }
  // (VEC: of a unit within the row)
  __device__ __forceinline__ Raw<T, VEC> get(int u) const {
    if constexpr (VEC) {
      const int l = threadIdx.x & 31;
      Raw<T, VEC> r;
#pragma unroll
      for (int h = 0; h < kHalves; ++h) {
        const int q = kHalves == 1 ? static_cast<int>(threadIdx.x)
                                   : 2 * (threadIdx.x - l) + ((2 * l + h) ^ ((l >> 2) & 1));
        const uint4 v = at[u * kHalves * kBlockThreads + q];
        r.w[4 * h] = v.x, r.w[4 * h + 1] = v.y, r.w[4 * h + 2] = v.z, r.w[4 * h + 3] = v.w;
      }
      return r;
    } else {
      return held[u];
    }
  }
};

// Parameters of a thread's units: in registers where they fit, else from L1.
template <int NV, bool HELD>
struct Weights {
  F2 held[HELD ? NV : 1][4];
  template <typename F>
  __device__ __forceinline__ void fetch(F&& make) {
    if constexpr (HELD) {
#pragma unroll
      for (int u = 0; u < NV; ++u) make(u, held[u]);
    }
  }
  template <typename F>
  __device__ __forceinline__ void get(F&& make, int u, F2 (&v)[4]) const {
    if constexpr (HELD) {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = held[u][i];
    } else {
      make(u, v);
    }
  }
};

constexpr int kRing = 3;                    // rows of a group in the ring, at most
constexpr size_t kBlockSmem = 220 * 1024;   // shared memory that the ring may take

// Waits until the copies of the oldest of `ring` rows under way are there.
__device__ __forceinline__ void ring_wait(int ring) {
  if (ring >= 3) copies_wait<2>();
  else if (ring == 2) copies_wait<1>();
  else copies_wait<0>();
  __syncwarp();   // the warp's copies, its other threads' among them
}

// Lets a kernel take the ring's shared memory, once for each device (`done`:
// the kernel's own, a bit a device).
inline cudaError_t allow_ring(const void* kernel, std::atomic<uint64_t>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           static_cast<int>(kBlockSmem));
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

// Blocks whose partial sums the backward's workspace has room for.
constexpr int kBlockBwdMaxParts = 160;

// What a token's gate gives, read a row ahead of its use.
__device__ __forceinline__ float token_gate(const BlockArgs& p, int t) {
  return p.gate == MOE_GATE_TOKEN && t < p.T ? *row_ptr<const float>(p.gate_rows, t) : 1.0f;
}

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
