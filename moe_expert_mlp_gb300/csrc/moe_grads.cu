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
// Nothing is added by atomics: equal gradients give equal bits.
#include <cuda_bf16.h>
#include <math.h>

#include "moe_internal.h"
#include "moe_ptx.cuh"

namespace moe {
namespace {

constexpr int kThreads = 512;
constexpr int kTile = 16384;        // elements of a tile
constexpr int kMaxList = 448;       // tensors of a launch: 28 KB of parameters
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

// Sum of the squares of 32 elements.  fp32 holds it unless it overflows or
// squares have vanished; then it is taken in fp64 (elements that are all zero
// need neither).
__device__ __forceinline__ double squares32(const float (&v)[32]) {
  float s = 0.0f;
#pragma unroll
  for (int e = 0; e < 32; ++e) s += v[e] * v[e];
  if (s >= 1e-30f && s <= 3e38f) return s;
  double d = 0.0;
  uint32_t any = 0;
#pragma unroll
  for (int e = 0; e < 32; ++e) any |= __float_as_uint(v[e]) << 1;
  if (any != 0) {
#pragma unroll 1
    for (int e = 0; e < 32; ++e) d += static_cast<double>(v[e]) * v[e];
  }
  return d;
}

template <bool INF>
struct Sum {
  double sum = 0.0;
  uint32_t top = 0;   // bits of the largest magnitude: NaN above Inf above the finite
  __device__ __forceinline__ void add(const float (&v)[32]) {
    if constexpr (INF) {
#pragma unroll
      for (int e = 0; e < 32; ++e) top = max(top, __float_as_uint(v[e]) & 0x7FFFFFFFu);
    } else {
      sum += squares32(v);
    }
  }
};

__device__ __forceinline__ float element(const char* base, long long i, bool f32) {
  return f32 ? reinterpret_cast<const float*>(base)[i]
             : __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(base)[i]);
}

// 8 elements from a 16-byte aligned place.
__device__ __forceinline__ void eight(const char* base, long long i, bool f32, float* v) {
  if (f32) {
    const float4* q = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(base) + i);
    const float4 a = q[0], b = q[1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  } else {
    const uint4 w = *reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(base) + i);
    v[0] = bf16_lo(w.x), v[1] = bf16_hi(w.x), v[2] = bf16_lo(w.y), v[3] = bf16_hi(w.y);
    v[4] = bf16_lo(w.z), v[5] = bf16_hi(w.z), v[6] = bf16_lo(w.w), v[7] = bf16_hi(w.w);
  }
}

// Whether rows are adjacent, so that a tile is one run of elements.
__device__ __forceinline__ bool one_run(const Tile& t, long long ld) {
  return t.rows == 1 || ld == t.cols;
}

template <bool INF>
__device__ __forceinline__ void add_tile(const Tensor& t, const Tile& q, Sum<INF>& s) {
  const int bytes = t.in32 ? 4 : 2;
  const int n = q.rows * q.cols;
  const char* base = t.in + (q.row * t.ld + q.col) * bytes;
  if (one_run(q, t.ld) && (reinterpret_cast<uintptr_t>(base) & 15) == 0) {
    for (int i = threadIdx.x * 8; i < n; i += kThreads * 32) {
      float v[32];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int at = i + u * kThreads * 8;
        if (at + 8 <= n) {
          eight(base, at, t.in32, v + 8 * u);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) v[8 * u + e] = at + e < n ? element(base, at + e, t.in32) : 0.0f;
        }
      }
      s.add(v);
    }
  } else {
    for (int i = threadIdx.x; i < n; i += kThreads * 32) {
      float v[32];
#pragma unroll
      for (int e = 0; e < 32; ++e) {
        const int at = i + e * kThreads;
        const int r = at / q.cols;
        v[e] = at < n ? element(base, r * t.ld + (at - r * q.cols), t.in32) : 0.0f;
      }
      s.add(v);
    }
  }
}

// Block sum (or maximum) of every thread's part, on thread 0.
template <bool INF>
__device__ __forceinline__ double block_total(const Sum<INF>& s, double* shared) {
  double v = INF ? static_cast<double>(s.top) : s.sum;   // the bits, exact in fp64
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const double w = __shfl_xor_sync(0xFFFFFFFFu, v, o);
    v = INF ? fmax(v, w) : v + w;
  }
  __syncthreads();
  if ((threadIdx.x & 31) == 0) shared[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.0;
  if (threadIdx.x == 0)
    for (int i = 0; i < static_cast<int>(blockDim.x) / 32; ++i)
      v = INF ? fmax(v, shared[i]) : v + shared[i];
  return v;
}

__device__ __forceinline__ int first_tile(int b, int blocks, int tiles) {
  return static_cast<int>(static_cast<long long>(b) * tiles / blocks);
}

template <bool INF, int N>
__global__ void __launch_bounds__(kThreads) k_grad_partials(const __grid_constant__ List<N> l,
                                                            double* __restrict__ part) {
  __shared__ double shared[kThreads / 32];
  const int begin = first_tile(blockIdx.x, gridDim.x, l.tiles);
  const int end = first_tile(blockIdx.x + 1, gridDim.x, l.tiles);
  int j = tensor_of(l, begin);
  if (threadIdx.x == 0 && blockIdx.x > 0 && j > 0 && l.t[j].first == begin)
    part[blockIdx.x + j - 1] = 0.0;   // the walk came from (block - 1, j - 1)
  for (int i = begin; i < end;) {
    const int stop = j + 1 < l.n ? min(end, l.t[j + 1].first) : end;
    Sum<INF> s;
    for (; i < stop; ++i) add_tile(l.t[j], tile_of(l.t[j], i - l.t[j].first), s);
    const double v = block_total(s, shared);
    if (threadIdx.x == 0) part[blockIdx.x + j] = v;
    ++j;
  }
}

__device__ __forceinline__ float norm_of(double v, bool inf) {
  return inf ? __uint_as_float(static_cast<uint32_t>(v)) : static_cast<float>(sqrt(v));
}

// One block: each tensor's norm from its slots (a warp each), and the total
// of this launch's slots into sums[at].
template <bool INF, int N>
__global__ void __launch_bounds__(1024) k_grad_join(const __grid_constant__ List<N> l, int blocks,
                                                    const double* __restrict__ part,
                                                    float* __restrict__ norms,
                                                    double* __restrict__ sums, int at, bool last,
                                                    float* __restrict__ norm) {
  __shared__ double shared[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (norms != nullptr) {
    for (int j = warp; j < l.n; j += 32) {
      // blocks whose runs meet tiles first .. next - 1
      const int first = l.t[j].first, next = j + 1 < l.n ? l.t[j + 1].first : l.tiles;
      int b = static_cast<int>(static_cast<long long>(first) * blocks / l.tiles);
      while (first_tile(b + 1, blocks, l.tiles) <= first) ++b;
      int e = static_cast<int>(static_cast<long long>(next - 1) * blocks / l.tiles);
      while (first_tile(e + 1, blocks, l.tiles) <= next - 1) ++e;
      double v = 0.0;
      for (int i = b + lane; i <= e; i += 32) v = INF ? fmax(v, part[i + j]) : v + part[i + j];
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const double w = __shfl_xor_sync(0xFFFFFFFFu, v, o);
        v = INF ? fmax(v, w) : v + w;
      }
      if (lane == 0) norms[l.t[j].id] = norm_of(v, INF);
    }
  }
  double v = 0.0;
  const int slots = l.n > 0 ? blocks + l.n - 1 : 0;
  for (int i = threadIdx.x; i < slots; i += 1024) v = INF ? fmax(v, part[i]) : v + part[i];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const double w = __shfl_xor_sync(0xFFFFFFFFu, v, o);
    v = INF ? fmax(v, w) : v + w;
  }
  if (lane == 0) shared[warp] = v;
  __syncthreads();
  if (threadIdx.x == 0) {
    double total = at > 0 ? sums[0] : 0.0;
    for (int i = 0; i < 32; ++i) total = INF ? fmax(total, shared[i]) : total + shared[i];
    sums[0] = total;
    if (last) norm[0] = norm_of(total, INF);
  }
}

__device__ __forceinline__ void put(char* base, long long i, bool f32, float v) {
  if (f32)
    reinterpret_cast<float*>(base)[i] = v;
  else
    reinterpret_cast<__nv_bfloat16*>(base)[i] = __float2bfloat16_rn(v);
}

template <int N>
__global__ void __launch_bounds__(kThreads) k_clip(const __grid_constant__ List<N> l,
                                                   const float* __restrict__ norm, float max_norm,
                                                   float eps) {
  float scale = max_norm / (*norm + eps);
  if (scale >= 1.0f) scale = 1.0f;       // a NaN stays
  const int begin = first_tile(blockIdx.x, gridDim.x, l.tiles);
  const int end = first_tile(blockIdx.x + 1, gridDim.x, l.tiles);
  int j = tensor_of(l, begin);
  for (int i = begin; i < end; ++i) {
    while (j + 1 < l.n && l.t[j + 1].first <= i) ++j;
    const Tensor& t = l.t[j];
    if (scale == 1.0f && t.in == t.out) continue;
    const Tile q = tile_of(t, i - t.first);
    const int n = q.rows * q.cols;
    const char* in = t.in + (q.row * t.ld + q.col) * (t.in32 ? 4 : 2);
    char* out = t.out + (q.row * t.ld_out + q.col) * (t.out32 ? 4 : 2);
    if (one_run(q, t.ld) && one_run(q, t.ld_out) &&
        ((reinterpret_cast<uintptr_t>(in) | reinterpret_cast<uintptr_t>(out)) & 15) == 0) {
#pragma unroll 4
      for (int at = threadIdx.x * 8; at < n; at += kThreads * 8) {
        float v[8];
        if (at + 8 <= n) {
          eight(in, at, t.in32, v);
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] *= scale;
          if (t.out32) {
            float4* to = reinterpret_cast<float4*>(reinterpret_cast<float*>(out) + at);
            to[0] = make_float4(v[0], v[1], v[2], v[3]);
            to[1] = make_float4(v[4], v[5], v[6], v[7]);
          } else {
            *reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(out) + at) =
                make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                           pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
          }
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
// last one taken (the list is full, or its tiles would pass 32 bits).
template <int N>
int fill(List<N>& l, const moe_grad_t* g, int from, int n) {
  l.n = 0;
  long long tiles = 0;
  int i = from;
  for (; i < n && l.n < N; ++i) {
    moe_grad_t q = g[i];
    if (q.rows == 0 || q.cols == 0) continue;
    const bool packed = q.rows == 1 || (q.ld == q.cols && (q.out == nullptr || q.ld_out == q.cols));
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
    t.out = static_cast<char*>(q.out);
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

template <int N, bool INF>
cudaError_t norm_pass(const moe_grad_t* g, int n, float* norm, float* norms, double* ws, int sms,
                      cudaStream_t s) {
  List<N> l;
  double* part = ws + 32;
  int from = 0;
  do {
    const int start = from;
    from = fill(l, g, from, n);
    const int blocks = min(l.tiles, min(4 * sms, kMaxBlocks));
    if (blocks > 0) k_grad_partials<INF, N><<<blocks, kThreads, 0, s>>>(l, part);
    k_grad_join<INF, N><<<1, 1024, 0, s>>>(l, blocks, part, norms, ws, start, from >= n, norm);
    const cudaError_t e = cudaGetLastError();
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
    from = fill(l, g, from, n);
    const int blocks = min(l.tiles, 4 * sms);
    if (blocks > 0) k_clip<N><<<blocks, kThreads, 0, s>>>(l, norm, max_norm, eps);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  } while (from < n);
  return cudaSuccess;
}

constexpr int kSmallList = 56;   // 3.6 KB of parameters

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
      n <= kSmallList ? clip_pass<kSmallList>(grads, n, norm, max_norm, eps, sms, stream)
                      : clip_pass<kMaxList>(grads, n, norm, max_norm, eps, sms, stream);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
