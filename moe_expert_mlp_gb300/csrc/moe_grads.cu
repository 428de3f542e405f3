// Global norm of a list of gradient tensors, and clipping.
//
// norm = sqrt(sum of squares) or the largest magnitude over every element of
// every tensor; out = g * min(1, max_norm / (norm + eps)).
//
// Bound by HBM: one or two operations an element.  The list travels in the
// kernel's parameters (no table on the device to go stale, nothing to copy),
// kMaxList tensors a launch.  Tensors are cut into tiles of kTile elements,
// and every block takes one contiguous run of the list's tiles, so that its
// partial sums are one for each tensor it meets: (block, tensor) pairs walk a
// staircase, pair (b, j) writes slot b + j, and a slot the walk jumps over is
// zeroed by the block behind it.  A second kernel adds the slots in order.
// Nothing is added by atomics: equal gradients, laid out alike and starting alike
// to 32 bytes, give equal bits on one GPU.
//
// Measured on 554 M bf16 gradients (64 experts of 2048 x 1408): norm 174 us =
// 6.4 TB/s (94 % of the rate of a copy), clipped into fp32 530 us = 6.3 TB/s;
// one call after the other 701 us, 93 % of the rate over the bytes of both
// passes.  The largest magnitude of the same list 163 us, its floor.  Small lists wait for their launches and last tiles: 84 fp32 tensors,
// 151 MB, 83 us for both, 81 % over the bytes of both passes.
#include <cuda_bf16.h>
#include <math.h>

#include <algorithm>

#include "moe_f2.cuh"
#include "moe_internal.h"
#include "moe_ptx.cuh"

namespace moe {
namespace {

constexpr int kThreads = 512;
constexpr int kTile = 16384;        // elements of a tile
constexpr int kMaxList = 448;       // tensors of a launch: 28 KB of parameters
constexpr int kResident = 2;        // blocks of an SM
constexpr int kMaxBlocks = 608;

struct Tensor {
  const char* in;
  char* out;
  long long rows, cols, ld, ld_out;
  int first;         // its first tile in the list
  int id;            // its place in the caller's list
  int in32, out32;   // fp32 (else bf16)
};

template <int N>
struct List {
  int n, tiles;      // tensors with elements, their tiles
  int each, more;    // tiles of a block; the first `more` blocks have one more
  Tensor t[N];
};

// Tiles of a tensor: pieces of rows at least kTile long, else whole rows
// together.
__host__ __device__ inline long long row_pieces(long long cols) {
  return cols >= kTile ? (cols + kTile - 1) / kTile : 1;
}
__host__ __device__ inline long long tile_rows(long long cols) {
  return cols >= kTile ? 1 : kTile / cols;
}

struct Tile {
  long long row, col;   // first element
  int rows, cols;
};

__device__ __forceinline__ Tile tile_of(const Tensor& t, int i) {
  Tile r;
  if (t.rows == 1) {   // without divisions
    r.row = 0;
    r.col = static_cast<long long>(i) * kTile;
    r.rows = 1;
    r.cols = static_cast<int>(min(static_cast<long long>(kTile), t.cols - r.col));
    return r;
  }
  const long long pieces = row_pieces(t.cols), many = tile_rows(t.cols);
  if (pieces > 1) {
    r.row = i / pieces;
    r.col = (i - r.row * pieces) * kTile;
    r.rows = 1;
    r.cols = static_cast<int>(min(static_cast<long long>(kTile), t.cols - r.col));
  } else {
    r.row = i * many;
    r.col = 0;
    r.rows = static_cast<int>(min(many, t.rows - r.row));
    r.cols = static_cast<int>(t.cols);
  }
  return r;
}

// Tensor of tile i.
template <int N>
__device__ __forceinline__ int tensor_of(const List<N>& l, int i) {
  int lo = 0, hi = l.n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (l.t[mid].first <= i) lo = mid; else hi = mid;
  }
  return lo;
}

__device__ __forceinline__ float element(const char* base, long long i, bool f32) {
  return f32 ? reinterpret_cast<const float*>(base)[i]
             : __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(base)[i]);
}

// 8 elements as they lie in memory: 4 words of bf16, 8 of fp32.
__device__ __forceinline__ void raw_eight(const char* base, int i, bool f32, uint32_t (&w)[8]) {
  if (f32) {
    load32_once(base + i * 4LL, w);
  } else {
    const uint4 q = *reinterpret_cast<const uint4*>(base + i * 2LL);
    w[0] = q.x, w[1] = q.y, w[2] = q.z, w[3] = q.w;
  }
}

// Whether a tile is one run of elements that starts on 32 bytes.
__device__ __forceinline__ bool wide_run(const Tile& t, const char* base, long long ld) {
  return (t.rows == 1 || ld == t.cols) && (reinterpret_cast<uintptr_t>(base) & 31) == 0;
}

// A thread's sum of squares over some tiles of a tensor, in eight fp32 chains
// of at most 16 squares each (kFlush tiles); then it goes to fp64.  The chains
// hold it unless they overflow or squares have vanished: then the caller takes
// it from the tiles again in fp64 (elements that are all zero need no second
// look).
constexpr int kFlush = 4;

struct Squares {
  F2 s[4];
  uint32_t any;   // the elements' bits but their signs
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < 4; ++i) s[i] = f2(0.0f);
    any = 0;
  }
  __device__ __forceinline__ void add(const uint32_t (&w)[8], bool f32) {
    if (f32) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const F2 v = f2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
        s[i] = fma2(v, v, s[i]);
        any |= (w[2 * i] | w[2 * i + 1]) & 0x7FFFFFFFu;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const F2 v = f2(bf16_lo(w[i]), bf16_hi(w[i]));
        s[i] = fma2(v, v, s[i]);
        any |= w[i] & 0x7FFF7FFFu;
      }
    }
  }
  __device__ __forceinline__ void add(const uint32_t (&w)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const F2 v = f2(bf16_lo(w[i]), bf16_hi(w[i]));
      s[i] = fma2(v, v, s[i]);
      any |= w[i] & 0x7FFF7FFFu;
    }
  }
  __device__ __forceinline__ void add(const uint32_t (&w)[8]) { add(w, true); }
  __device__ __forceinline__ void add(int i, float v) {
    const F2 q = i & 1 ? f2(0.0f, v) : f2(v, 0.0f);
    s[i / 2] = fma2(q, q, s[i / 2]);
    any |= __float_as_uint(v) & 0x7FFFFFFFu;
  }
  __device__ __forceinline__ float total() const { return sum((s[0] + s[1]) + (s[2] + s[3])); }
};

// The largest magnitude, as bits (NaN above Inf above the finite); bf16 pairs
// side by side.
struct Top {
  uint32_t top, pair;
  __device__ __forceinline__ void clear() { top = pair = 0; }
  __device__ __forceinline__ void add(const uint32_t (&w)[8], bool f32) {
    if (f32) {
#pragma unroll
      for (int i = 0; i < 8; ++i) top = max(top, w[i] & 0x7FFFFFFFu);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) pair = __vmaxu2(pair, w[i] & 0x7FFF7FFFu);
    }
  }
  __device__ __forceinline__ void add(int, float v) { top = max(top, __float_as_uint(v) & 0x7FFFFFFFu); }
  __device__ __forceinline__ uint32_t total() const {
    return max(top, max(pair << 16, pair & 0xFFFF0000u));
  }
};

// Hands a thread its elements of a tile: 8 at a time, or single ones with the
// chain they belong to.
template <typename Sum>
__device__ __forceinline__ void add_tile(const Tensor& t, const Tile& q, Sum& s) {
  const int n = q.rows * q.cols;
  const char* base = t.in + (q.row * t.ld + q.col) * (t.in32 ? 4 : 2);
  if (wide_run(q, base, t.ld)) {
    if (n == kTile) {
      // all four loads in flight
      uint32_t w[4][8];
      if (t.in32) {
#pragma unroll
        for (int u = 0; u < 4; ++u) raw_eight(base, (u * kThreads + threadIdx.x) * 8, true, w[u]);
#pragma unroll
        for (int u = 0; u < 4; ++u) s.add(w[u], true);
      } else {
#pragma unroll
        for (int u = 0; u < 4; ++u) raw_eight(base, (u * kThreads + threadIdx.x) * 8, false, w[u]);
#pragma unroll
        for (int u = 0; u < 4; ++u) s.add(w[u], false);
      }
      return;
    }
    for (int at = threadIdx.x * 8; at < n; at += kThreads * 8) {
      if (at + 8 <= n) {
        uint32_t w[8];
        raw_eight(base, at, t.in32, w);
        s.add(w, t.in32);
      } else {
        for (int e = 0; at + e < n; ++e) s.add(e, element(base, at + e, t.in32));
      }
    }
    return;
  }
  for (int at = threadIdx.x; at < n; at += kThreads) {
    const int r = at / q.cols;
    s.add((at / kThreads) & 7, element(base, r * t.ld + (at - r * q.cols), t.in32));
  }
}

// kFlush whole tiles on end, 128 bytes of a thread in flight at a time (with 64
// the loads' latency showed: 247 instead of 174 us over 1.1 GB of bf16).
template <bool IN32>
__device__ __forceinline__ void add_four(const char* base, Squares& s) {
  constexpr int kBatch = IN32 ? 4 : 8;
#pragma unroll
  for (int b = 0; b < 4 * kFlush / kBatch; ++b) {
    uint32_t w[kBatch][IN32 ? 8 : 4];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int at = ((b * kBatch + u) * kThreads + threadIdx.x) * 8;
      if constexpr (IN32) {
        load32_once(base + at * 4LL, w[u]);
      } else {
        const uint4 q = *reinterpret_cast<const uint4*>(base + at * 2LL);
        w[u][0] = q.x, w[u][1] = q.y, w[u][2] = q.z, w[u][3] = q.w;
      }
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) s.add(w[u]);
  }
}

// The squares of the same elements once more, in fp64 (out of the way: called
// only where fp32 does not hold them).
__device__ __noinline__ double squares_again(const Tensor& t, int from, int to) {
  double d = 0.0;
  for (int i = from; i < to; ++i) {
    const Tile q = tile_of(t, i);
    const int n = q.rows * q.cols;
    const char* base = t.in + (q.row * t.ld + q.col) * (t.in32 ? 4 : 2);
    const int step = wide_run(q, base, t.ld) ? 8 : 1;
    for (int at = threadIdx.x * step; at < n; at += kThreads * step)
      for (int e = 0; e < step && at + e < n; ++e) {
        const int r = (at + e) / q.cols;
        const double v = element(base, r * t.ld + (at + e - r * q.cols), t.in32);
        d += v * v;
      }
  }
  return d;
}

// A thread's part of tiles from .. to - 1 of a tensor: its squares, or the
// bits of its largest magnitude (exact in fp64).
template <bool INF>
__device__ __forceinline__ double add_tiles(const Tensor& t, int from, int to) {
  if constexpr (INF) {
    Top s;
    s.clear();
    for (int i = from; i < to; ++i) add_tile(t, tile_of(t, i), s);
    return static_cast<double>(s.total());
  } else {
    double d = 0.0;
    const bool whole = t.rows == 1 && (reinterpret_cast<uintptr_t>(t.in) & 31) == 0;
    for (int i = from; i < to; i += kFlush) {
      const int stop = min(i + kFlush, to);
      Squares s;
      s.clear();
      if (whole && (i + kFlush) * static_cast<long long>(kTile) <= t.cols && stop - i == kFlush)
        t.in32 ? add_four<true>(t.in + i * (kTile * 4LL), s)
               : add_four<false>(t.in + i * (kTile * 2LL), s);
      else
        for (int k = i; k < stop; ++k) add_tile(t, tile_of(t, k), s);
      const float v = s.total();
      if (v >= 1e-30f && v <= 3e38f)
        d += v;
      else if (s.any != 0)
        d += squares_again(t, i, stop);
    }
    return d;
  }
}

// Block sum (or maximum) of every thread's part, on thread 0.
template <bool INF>
__device__ __forceinline__ double block_total(double v, double* shared) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const double w = __shfl_xor_sync(0xFFFFFFFFu, v, o);
    v = INF ? fmax(v, w) : v + w;
  }
  __syncthreads();
  if ((threadIdx.x & 31) == 0) shared[threadIdx.x >> 5] = v;
  __syncthreads();
  if (threadIdx.x >= 32) return 0.0;
  v = threadIdx.x < kThreads / 32 ? shared[threadIdx.x] : 0.0;
#pragma unroll
  for (int o = kThreads / 64; o > 0; o >>= 1) {
    const double w = __shfl_xor_sync(0xFFFFFFFFu, v, o);
    v = INF ? fmax(v, w) : v + w;
  }
  return v;
}

// The block's run of tiles, and the block of a tile.
template <int N>
__device__ __forceinline__ int first_tile(const List<N>& l, int b) {
  return b * l.each + min(b, l.more);
}
template <int N>
__device__ __forceinline__ int block_of(const List<N>& l, int i) {
  const int wide = l.more * (l.each + 1);
  return i < wide ? i / (l.each + 1) : l.more + (i - wide) / l.each;
}

template <bool INF, int N>
__global__ void __launch_bounds__(kThreads, kResident) k_grad_partials(const __grid_constant__ List<N> l,
                                                            double* __restrict__ part) {
  __shared__ double shared[kThreads / 32];
  const int begin = first_tile(l, blockIdx.x);
  const int end = first_tile(l, blockIdx.x + 1);
  int j = tensor_of(l, begin);
  if (threadIdx.x == 0 && blockIdx.x > 0 && j > 0 && l.t[j].first == begin)
    part[blockIdx.x + j - 1] = 0.0;   // the walk came from (block - 1, j - 1)
  for (int i = begin; i < end;) {
    const int stop = j + 1 < l.n ? min(end, l.t[j + 1].first) : end;
    const double v = block_total<INF>(
        add_tiles<INF>(l.t[j], i - l.t[j].first, stop - l.t[j].first), shared);
    if (threadIdx.x == 0) part[blockIdx.x + j] = v;
    i = stop;
    ++j;
  }
}

__device__ __forceinline__ float norm_of(double v, bool inf) {
  return inf ? __uint_as_float(static_cast<uint32_t>(v)) : static_cast<float>(sqrt(v));
}

template <bool INF>
__device__ __forceinline__ double warp_total(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const double w = __shfl_xor_sync(0xFFFFFFFFu, v, o);
    v = INF ? fmax(v, w) : v + w;
  }
  return v;
}

// Block 0: the total of this launch's slots into sums[0], added to the launches'
// before it.  Blocks behind it: tensors' norms, a warp each.  Started while
// k_grad_partials still runs (programmatic launch), waits for its end.
template <bool INF, int N>
__global__ void __launch_bounds__(1024) k_grad_join(const __grid_constant__ List<N> l, int blocks,
                                                    const double* __restrict__ part,
                                                    float* __restrict__ norms,
                                                    double* __restrict__ sums, bool first,
                                                    bool last, float* __restrict__ norm) {
  __shared__ double shared[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (blockIdx.x > 0) {
    const int j = (blockIdx.x - 1) * 32 + warp;
    if (j >= l.n) return;
    const int next = j + 1 < l.n ? l.t[j + 1].first : l.tiles;
    const int b = block_of(l, l.t[j].first), e = block_of(l, next - 1);
    wait_for_previous();
    double v = 0.0;
    for (int i = b + lane; i <= e; i += 32) v = INF ? fmax(v, part[i + j]) : v + part[i + j];
    v = warp_total<INF>(v);
    if (lane == 0) norms[l.t[j].id] = norm_of(v, INF);
    return;
  }
  wait_for_previous();
  double v = 0.0;
  const int slots = l.n > 0 ? blocks + l.n - 1 : 0;
  for (int i = threadIdx.x; i < slots; i += 1024) v = INF ? fmax(v, part[i]) : v + part[i];
  v = warp_total<INF>(v);
  if (lane == 0) shared[warp] = v;
  __syncthreads();
  if (warp == 0) {
    v = warp_total<INF>(shared[lane]);
    if (lane == 0) {
      if (!first) v = INF ? fmax(sums[0], v) : sums[0] + v;
      sums[0] = v;
      if (last) norm[0] = norm_of(v, INF);
    }
  }
}

__device__ __forceinline__ void put(char* base, long long i, bool f32, float v) {
  if (f32)
    reinterpret_cast<float*>(base)[i] = v;
  else
    reinterpret_cast<__nv_bfloat16*>(base)[i] = __float2bfloat16_rn(v);
}

// 8 elements, scaled.
__device__ __forceinline__ void put_eight(char* out, int i, bool out32, const uint32_t (&w)[8],
                                          bool in32, float scale) {
  float v[8];
#pragma unroll
  for (int e = 0; e < 8; ++e)
    v[e] = scale * (in32 ? __uint_as_float(w[e]) : e & 1 ? bf16_hi(w[e / 2]) : bf16_lo(w[e / 2]));
  if (out32)
    store32(out + i * 4LL, v);
  else
    *reinterpret_cast<uint4*>(out + i * 2LL) =
        make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                   pack_bf16x2(v[6], v[7]));
}

template <bool IN32, bool OUT32>
__device__ __forceinline__ void clip_whole_tile(const char* in, char* out, float scale) {
  uint32_t w[4][8];
#pragma unroll
  for (int u = 0; u < 4; ++u) raw_eight(in, (u * kThreads + threadIdx.x) * 8, IN32, w[u]);
#pragma unroll
  for (int u = 0; u < 4; ++u)
    put_eight(out, (u * kThreads + threadIdx.x) * 8, OUT32, w[u], IN32, scale);
}

// The blocks take the runs of tiles that they take in k_grad_partials (other ones
// where a contiguous gradient's out is not contiguous) and walk them backwards:
// what that kernel read last is read first, while L2 has it.
template <int N>
__global__ void __launch_bounds__(kThreads, kResident) k_clip(const __grid_constant__ List<N> l,
                                                              const float* __restrict__ norm,
                                                              float max_norm, float eps) {
  wait_for_previous();                   // programmatic launch: the norm is there
  float scale = max_norm / (*norm + eps);
  if (scale >= 1.0f) scale = 1.0f;       // a NaN stays
  const int begin = first_tile(l, blockIdx.x);
  const int end = first_tile(l, blockIdx.x + 1);
  int j = tensor_of(l, end - 1);
  for (int i = end - 1; i >= begin; --i) {
    while (l.t[j].first > i) --j;
    const Tensor& t = l.t[j];
    if (scale == 1.0f && t.in == t.out) continue;
    const Tile q = tile_of(t, i - t.first);
    const int n = q.rows * q.cols;
    const char* in = t.in + (q.row * t.ld + q.col) * (t.in32 ? 4 : 2);
    char* out = t.out + (q.row * t.ld_out + q.col) * (t.out32 ? 4 : 2);
    if (wide_run(q, in, t.ld) && wide_run(q, out, t.ld_out)) {
      if (n == kTile) {
        if (t.in32)
          t.out32 ? clip_whole_tile<true, true>(in, out, scale)
                  : clip_whole_tile<true, false>(in, out, scale);
        else
          t.out32 ? clip_whole_tile<false, true>(in, out, scale)
                  : clip_whole_tile<false, false>(in, out, scale);
        continue;
      }
      for (int at = threadIdx.x * 8; at < n; at += kThreads * 8) {
        if (at + 8 <= n) {
          uint32_t w[8];
          raw_eight(in, at, t.in32, w);
          put_eight(out, at, t.out32, w, t.in32, scale);
        } else {
          for (int e = 0; at + e < n; ++e)
            put(out, at + e, t.out32, element(in, at + e, t.in32) * scale);
        }
      }
    } else {
      for (int at = threadIdx.x; at < n; at += kThreads) {
        const int r = at / q.cols, c = at - r * q.cols;
        put(out, r * t.ld_out + c, t.out32, element(in, r * t.ld + c, t.in32) * scale);
      }
    }
  }
}

bool known(int t) { return t == MOE_DTYPE_BF16 || t == MOE_DTYPE_FP32; }
int bytes_of(int t) { return t == MOE_DTYPE_FP32 ? 4 : 2; }

moe_status_t check_grad(const moe_grad_t& g, bool clip) {
  if (!known(g.dtype) || (clip && !known(g.out_dtype))) return MOE_ERR_UNSUPPORTED;
  if (g.rows < 0 || g.cols < 0) return MOE_ERR_SHAPE;
  if (g.rows == 0 || g.cols == 0) return MOE_OK;
  if (!g.grad || (clip && !g.out)) return MOE_ERR_NULL;
  constexpr long long most = 1LL << 40;
  if (g.rows > most || g.cols > most || g.rows > most / g.cols) return MOE_ERR_SHAPE;
  if (g.rows > 1 && (g.ld < g.cols || (clip && g.ld_out < g.cols))) return MOE_ERR_SHAPE;
  if (reinterpret_cast<uintptr_t>(g.grad) % bytes_of(g.dtype)) return MOE_ERR_SHAPE;
  if (clip) {
    if (reinterpret_cast<uintptr_t>(g.out) % bytes_of(g.out_dtype)) return MOE_ERR_SHAPE;
    // in place: the same elements
    if (g.grad == g.out && (g.dtype != g.out_dtype || (g.rows > 1 && g.ld != g.ld_out)))
      return MOE_ERR_UNSUPPORTED;
  }
  return MOE_OK;
}

// Appends tensors from the list's place `from`; returns the place behind the
// last one taken (the list is full, or its tiles would pass 32 bits).  Without
// `clip` nothing is asked of the outs, which the caller may not have set.
template <int N>
int fill(List<N>& l, const moe_grad_t* g, int from, int n, bool clip) {
  l.n = 0;
  long long tiles = 0;
  int i = from;
  for (; i < n && l.n < N; ++i) {
    moe_grad_t q = g[i];
    if (q.rows == 0 || q.cols == 0) continue;
    const bool packed = q.rows == 1 || (q.ld == q.cols && (!clip || q.ld_out == q.cols));
    if (packed) {
      q.cols *= q.rows;
      q.rows = 1;
      q.ld = q.ld_out = q.cols;
    }
    const long long count = q.cols >= kTile
                                ? q.rows * row_pieces(q.cols)
                                : (q.rows + tile_rows(q.cols) - 1) / tile_rows(q.cols);
    if (tiles + count > 0x7FFFFFFFLL / 2) break;
    Tensor& t = l.t[l.n++];
    t.in = static_cast<const char*>(q.grad);
    t.out = clip ? static_cast<char*>(q.out) : nullptr;
    t.rows = q.rows;
    t.cols = q.cols;
    t.ld = q.ld;
    t.ld_out = q.ld_out;
    t.first = static_cast<int>(tiles);
    t.id = i;
    t.in32 = q.dtype == MOE_DTYPE_FP32;
    t.out32 = q.out_dtype == MOE_DTYPE_FP32;
    tiles += count;
  }
  l.tiles = static_cast<int>(tiles);
  return i;
}

// Shares the tiles among the resident blocks; returns their number.
template <int N>
int share(List<N>& l, int sms) {
  const int blocks = std::min(l.tiles, std::min(kResident * sms, kMaxBlocks));
  l.each = blocks > 0 ? l.tiles / blocks : 0;
  l.more = blocks > 0 ? l.tiles % blocks : 0;
  return blocks;
}

template <int N, bool INF>
cudaError_t norm_pass(const moe_grad_t* g, int n, float* norm, float* norms, double* ws, int sms,
                      cudaStream_t s) {
  List<N> l;
  double* part = ws + 32;
  int from = 0;
  do {
    const int start = from;
    from = fill(l, g, from, n, false);
    const int blocks = share(l, sms);
    if (blocks > 0) k_grad_partials<INF, N><<<blocks, kThreads, 0, s>>>(l, part);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const int joins = norms != nullptr ? 1 + (l.n + 31) / 32 : 1;
    e = launch_dependent(k_grad_join<INF, N>, joins, 1024, s, l, blocks,
                         static_cast<const double*>(part), norms, ws, start == 0, from >= n, norm);
    if (e != cudaSuccess) return e;
  } while (from < n);
  return cudaSuccess;
}

template <int N>
cudaError_t clip_pass(const moe_grad_t* g, int n, const float* norm, float max_norm, float eps,
                      int sms, cudaStream_t s) {
  List<N> l;
  int from = 0;
  do {
    from = fill(l, g, from, n, true);
    const int blocks = share(l, sms);
    if (blocks == 0) continue;
    const cudaError_t e = launch_dependent(k_clip<N>, blocks, kThreads, s, l, norm, max_norm, eps);
    if (e != cudaSuccess) return e;
  } while (from < n);
  return cudaSuccess;
}

// Lists of up to so many tensors: 3.6 and 10 KB of parameters.
constexpr int kSmallList = 56, kMiddleList = 160;

size_t norm_ws_bytes() { return (32 + kMaxBlocks + kMaxList) * sizeof(double); }

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

moe_status_t moe_grad_norm_workspace_size(int32_t n, size_t* bytes) {
  if (!bytes) return MOE_ERR_NULL;
  if (n < 0) return MOE_ERR_SHAPE;
  *bytes = norm_ws_bytes();
  return MOE_OK;
}

moe_status_t moe_grad_norm(const moe_grad_t* grads, int32_t n, int32_t norm_type, float* norm,
                           float* norms, void* ws, size_t ws_bytes, cudaStream_t stream) {
  if (n < 0) return MOE_ERR_SHAPE;
  if ((n > 0 && !grads) || !norm || !ws) return MOE_ERR_NULL;
  if (norm_type != MOE_GRAD_NORM_L2 && norm_type != MOE_GRAD_NORM_INF) return MOE_ERR_UNSUPPORTED;
  bool empty = false;
  for (int i = 0; i < n; ++i) {
    const moe_status_t st = check_grad(grads[i], false);
    if (st != MOE_OK) return st;
    empty = empty || grads[i].rows == 0 || grads[i].cols == 0;
  }
  if (reinterpret_cast<uintptr_t>(ws) % 16 || reinterpret_cast<uintptr_t>(norm) % 4 ||
      reinterpret_cast<uintptr_t>(norms) % 4)
    return MOE_ERR_SHAPE;
  if (ws_bytes < norm_ws_bytes()) return MOE_ERR_WORKSPACE;
  int sms, *status;
  const moe_status_t st = current_device(&sms, &status);
  if (st != MOE_OK) return st;
  if (norms && empty && cudaMemsetAsync(norms, 0, sizeof(float) * n, stream) != cudaSuccess)
    return MOE_ERR_CUDA;
  double* w = static_cast<double*>(ws);
  const bool inf = norm_type == MOE_GRAD_NORM_INF;
  cudaError_t e;
  if (n <= kSmallList)
    e = inf ? norm_pass<kSmallList, true>(grads, n, norm, norms, w, sms, stream)
            : norm_pass<kSmallList, false>(grads, n, norm, norms, w, sms, stream);
  else if (n <= kMiddleList)
    e = inf ? norm_pass<kMiddleList, true>(grads, n, norm, norms, w, sms, stream)
            : norm_pass<kMiddleList, false>(grads, n, norm, norms, w, sms, stream);
  else
    e = inf ? norm_pass<kMaxList, true>(grads, n, norm, norms, w, sms, stream)
            : norm_pass<kMaxList, false>(grads, n, norm, norms, w, sms, stream);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

moe_status_t moe_clip_grads(const moe_grad_t* grads, int32_t n, const float* norm, float max_norm,
                            float eps, cudaStream_t stream) {
  if (n < 0) return MOE_ERR_SHAPE;
  if ((n > 0 && !grads) || !norm) return MOE_ERR_NULL;
  if (!(max_norm >= 0.0f) || !(eps >= 0.0f) || !isfinite(max_norm) || !isfinite(eps))
    return MOE_ERR_SHAPE;
  for (int i = 0; i < n; ++i) {
    const moe_status_t st = check_grad(grads[i], true);
    if (st != MOE_OK) return st;
  }
  if (reinterpret_cast<uintptr_t>(norm) % 4) return MOE_ERR_SHAPE;
  int sms, *status;
  const moe_status_t st = current_device(&sms, &status);
  if (st != MOE_OK) return st;
  const cudaError_t e =
      n <= kSmallList    ? clip_pass<kSmallList>(grads, n, norm, max_norm, eps, sms, stream)
      : n <= kMiddleList ? clip_pass<kMiddleList>(grads, n, norm, max_norm, eps, sms, stream)
                         : clip_pass<kMaxList>(grads, n, norm, max_norm, eps, sms, stream);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
