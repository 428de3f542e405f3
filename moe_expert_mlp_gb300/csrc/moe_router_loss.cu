// The router's losses and their gradient (see include/moe.h for the formulas).
//
// Both passes are one read of the logits: a token's row lies in the registers
// of a group of 8 or 32 lanes, whose exchanges give its maximum, its sum of
// exponentials and, in the backward, <f, p>; the next token's row is on its way
// meanwhile.  What they cannot do without is that read (and the backward's
// write); the arithmetic, one exponential an element, is below it.
//
// Forward: the tokens are cut into chunks of equal length, one block each, and
// a chunk at the ends of sequences into segments.  Chunks and sequences both
// ascend, so the segment of chunk c and sequence s has the number c + s to
// itself.  A block writes its segments' sums of p, counts and squares, and the
// segments of a sequence are added up in ascending order, so the result does
// not depend on the order in which blocks ran: by a second launch, or, with no
// more chunks than a cluster has blocks, by the cluster that made them.
#include <math.h>

#include "moe_internal.h"
#include "moe_ptx.cuh"

namespace moe {
namespace {

constexpr int kFwdThreads = 1024;
constexpr int kBwdThreads = 256;
constexpr int kFwdMostTokens = 1024;  // of a chunk: 32 of a warp are added in fp32 one by one
constexpr int kLossCluster = 8;       // chunks that one launch makes and joins

struct LossArgs {
  const float* logits;
  const int32_t* topk_idx;
  const uint8_t* mask;         // [T] or null: every token counts
  const int32_t* seq_offsets;  // [S+1] or null: one sequence of all tokens
  int32_t* counts;             // [S,E]
  int32_t* tokens;             // [S+1]
  float* probs;                // [S,E]
  float* loss;                 // [3]
  const float* dloss;          // backward: null = 1
  const float* dw;             // backward: null = no share of the weights
  const float* topk_w;
  float* dlogits;
  // workspace: per segment, and per (sequence, 32 experts)
  float* seg_p;                // [segments, E]
  int32_t* seg_count;          // [segments, E]
  float* seg_z;                // [segments]
  int32_t* seg_tokens;         // [segments]
  float* term;                 // [S, e_blocks]: sum of count * P over 32 experts
  unsigned int* done;
  int* status;
  int T, E, k, S, chunk, chunks;
  float balance, z;
};

// Element j, i of a lane's share of a row: VEC consecutive experts at a time.
template <int LANES, int VEC>
__device__ __forceinline__ int expert_of(int lane, int j) {
  return (j * LANES + lane) * VEC;
}

template <int LANES>
__device__ __forceinline__ uint32_t group_lanes() {
  if constexpr (LANES == 32)
    return 0xFFFFFFFFu;
  else
    return ((1u << LANES) - 1u) << (threadIdx.x % 32 / LANES * LANES);
}

template <int LANES>
__device__ __forceinline__ float group_max(float v, uint32_t mask) {
  if constexpr (LANES == 32) {
    asm volatile("redux.sync.max.f32 %0, %0, %1;" : "+f"(v) : "r"(mask));
  } else {
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(mask, v, o));
  }
  return v;
}

template <int LANES>
__device__ __forceinline__ float group_sum(float v, uint32_t mask) {
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) v += __shfl_xor_sync(mask, v, o);
  return v;
}

// Softmax of one row over the group's lanes: x becomes exp(x - top), inv the
// reciprocal of their sum, and with DOT dot is <f, p>.  Returns logsumexp.  A row
// without a logit above -inf has p = 0 and gives 0.  (The maxima pass over NaN,
// which then reaches the sum.)
template <int LANES, int N, bool DOT>
__device__ __forceinline__ float row_softmax(float (&x)[N], float& inv, const float* f, float& dot,
                                             uint32_t mask) {
  float top = x[0];
#pragma unroll
  for (int i = 1; i < N; ++i) top = fmaxf(top, x[i]);
  top = group_max<LANES>(top, mask);
  float sum = 0.0f;
  dot = 0.0f;
  if (top == -INFINITY) {
    bool nan = false;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      nan = nan || x[i] != x[i];
      x[i] = 0.0f;
    }
    inv = __any_sync(mask, nan) ? __int_as_float(0x7FC00000) : 0.0f;
    dot = inv;
    return inv;
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    x[i] = __expf(x[i] - top);
    sum += x[i];
    if constexpr (DOT) dot = fmaf(f[i], x[i], dot);
  }
  sum = group_sum<LANES>(sum, mask);
  inv = 1.0f / sum;
  if constexpr (DOT) dot = group_sum<LANES>(dot, mask) * inv;
  return top + logf(sum);
}

// A lane's share of a row of floats; `fill` past the experts.
template <int LANES, int N, int VEC>
__device__ __forceinline__ void load_row(const float* row, int E, int lane, float fill,
                                         float (&x)[N]) {
#pragma unroll
  for (int j = 0; j < N / VEC; ++j) {
    const int e = expert_of<LANES, VEC>(lane, j);
    if constexpr (VEC == 4) {
      const float4 v = e < E ? __ldg(reinterpret_cast<const float4*>(row + e))
                             : make_float4(fill, fill, fill, fill);
      x[4 * j] = v.x;
      x[4 * j + 1] = v.y;
      x[4 * j + 2] = v.z;
      x[4 * j + 3] = v.w;
    } else {
      x[j] = e < E ? __ldg(row + e) : fill;
    }
  }
}

// First sequence whose end lies behind token t (S when none does).
__device__ __forceinline__ int sequence_of(const LossArgs& a, int t) {
  if (a.seq_offsets == nullptr) return t < a.T ? 0 : a.S;
  int lo = 0, hi = a.S;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(a.seq_offsets + mid + 1) > t) hi = mid; else lo = mid + 1;
  }
  return lo;
}

__device__ __forceinline__ void sequence_span(const LossArgs& a, int s, int* begin, int* end) {
  if (a.seq_offsets == nullptr) {
    *begin = 0;
    *end = a.T;
    return;
  }
  *begin = max(__ldg(a.seq_offsets + s), 0);
  *end = min(__ldg(a.seq_offsets + s + 1), a.T);
}

template <typename V>
__device__ __forceinline__ V warp_sum(V v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

// What a block sums up with, all but `part` a value a warp.
struct LossShared {
  float p[32][kMaxExperts];      // a row of each warp
  float part[4][kMaxExperts];
  int count[kMaxExperts];
  float z[32];
  int n[32];
};

// A block's segments: sums of p, counts, squares and tokens of chunk c.
template <int LANES, int N, int VEC>
__device__ __forceinline__ void chunk_segments(const LossArgs& a, int c, LossShared& sh) {
  constexpr int kGroups = kFwdThreads / LANES;
  const int group = threadIdx.x / LANES, lane = threadIdx.x % LANES;
  const int warp = threadIdx.x >> 5;
  const uint32_t mask = group_lanes<LANES>();
  const int t0 = c * a.chunk, t1 = min(t0 + a.chunk, a.T);
  for (int s = sequence_of(a, t0); s < a.S; ++s) {
    int begin, end;
    sequence_span(a, s, &begin, &end);
    if (begin >= t1) break;
    begin = max(begin, t0);
    end = min(end, t1);
    if (begin >= end) continue;
    if (threadIdx.x < kMaxExperts) sh.count[threadIdx.x] = 0;
    float acc[N], next[N], z = 0.0f;
    int n = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) acc[i] = next[i] = 0.0f;
    const float* row = a.logits + static_cast<long long>(begin + group) * a.E;
    bool live = false;
    if (begin + group < end) {
      load_row<LANES, N, VEC>(row, a.E, lane, -INFINITY, next);
      live = a.mask == nullptr || a.mask[begin + group] != 0;
    }
    __syncthreads();
    // the experts' counts meanwhile
    for (int i = threadIdx.x; i < (end - begin) * a.k; i += kFwdThreads) {
      if (a.mask != nullptr && a.mask[begin + i / a.k] == 0) continue;
      const int e = __ldg(a.topk_idx + static_cast<long long>(begin) * a.k + i);
      if (e < 0 || e >= a.E) set_status(a.status, MOE_DEV_BAD_EXPERT);
      else atomicAdd(&sh.count[e], 1);
    }
    for (int t = begin + group; t < end; t += kGroups) {
      float x[N], inv, unused;
#pragma unroll
      for (int i = 0; i < N; ++i) x[i] = next[i];
      const bool counted = live;
      row += static_cast<long long>(kGroups) * a.E;
      if (t + kGroups < end) {
        load_row<LANES, N, VEC>(row, a.E, lane, -INFINITY, next);
        live = a.mask == nullptr || a.mask[t + kGroups] != 0;
      }
      if (!counted) continue;
      const float lse = row_softmax<LANES, N, false>(x, inv, nullptr, unused, mask);
#pragma unroll
      for (int i = 0; i < N; ++i) acc[i] = fmaf(x[i], inv, acc[i]);
      z = fmaf(lse, lse, z);
      ++n;
    }
    __syncwarp();
    // the groups of a warp, then the warps
#pragma unroll
    for (int o = LANES; o < 32; o <<= 1) {
#pragma unroll
      for (int i = 0; i < N; ++i) acc[i] += __shfl_xor_sync(0xFFFFFFFFu, acc[i], o);
      z += __shfl_xor_sync(0xFFFFFFFFu, z, o);
      n += __shfl_xor_sync(0xFFFFFFFFu, n, o);
    }
    if (threadIdx.x % 32 < LANES) {
#pragma unroll
      for (int j = 0; j < N / VEC; ++j)
#pragma unroll
        for (int i = 0; i < VEC; ++i)
          sh.p[warp][expert_of<LANES, VEC>(lane, j) + i] = acc[j * VEC + i];
      if (lane == 0) {
        sh.z[warp] = z;
        sh.n[warp] = n;
      }
    }
    __syncthreads();
    const long long seg = static_cast<long long>(c) + s;
    const int e = threadIdx.x % kMaxExperts, q = threadIdx.x / kMaxExperts;
    if (e < a.E) {
      float p = 0.0f;
#pragma unroll
      for (int w = 0; w < 8; ++w) p += sh.p[8 * q + w][e];
      sh.part[q][e] = p;
    }
    __syncthreads();
    if (q == 0 && e < a.E) {
      a.seg_p[seg * a.E + e] = (sh.part[0][e] + sh.part[1][e]) + (sh.part[2][e] + sh.part[3][e]);
      a.seg_count[seg * a.E + e] = sh.count[e];
    }
    if (warp == 31) {
      const float zz = warp_sum(sh.z[threadIdx.x & 31]);
      const int nn = warp_sum(sh.n[threadIdx.x & 31]);
      if (threadIdx.x % 32 == 0) {
        a.seg_z[seg] = zz;
        a.seg_tokens[seg] = nn;
      }
    }
    __syncthreads();
  }
}

// 32 experts (block eb of blocks) of sequence s: their segments' sums over the
// block's 32 warps.
__device__ __forceinline__ void join_sequence(const LossArgs& a, int s, int eb, int blocks,
                                              float (*s_p)[33], int (*s_c)[33], int* s_n) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int e = eb * 32 + lane;
  int begin, end;
  sequence_span(a, s, &begin, &end);
  const int c0 = begin / a.chunk, c1 = end > begin ? (end - 1) / a.chunk + 1 : c0;
  float p = 0.0f;
  int count = 0, n = 0;
#pragma unroll 4
  for (int c = c0 + warp; c < c1; c += 32) {
    const long long seg = static_cast<long long>(c) + s;
    if (e < a.E) {
      p += __ldcg(a.seg_p + seg * a.E + e);
      count += __ldcg(a.seg_count + seg * a.E + e);
    }
    n += __ldcg(a.seg_tokens + seg);
  }
  s_p[warp][lane] = p;
  s_c[warp][lane] = count;
  if (lane == 0) s_n[warp] = n;
  __syncthreads();
  // a warp an expert, its lanes the 32 sums
  p = warp_sum(s_p[lane][warp]);
  count = warp_sum(s_c[lane][warp]);
  n = warp_sum(s_n[lane]);
  __syncthreads();
  const float mean = n > 0 ? p / static_cast<float>(n) : 0.0f;
  if (lane == 0) {
    const int mine = eb * 32 + warp;
    if (mine < a.E) {
      a.probs[static_cast<long long>(s) * a.E + mine] = mean;
      a.counts[static_cast<long long>(s) * a.E + mine] = count;
    }
    // N_s f P = E / k * count * P
    s_p[0][warp] = mine < a.E ? static_cast<float>(count) * mean : 0.0f;
  }
  __syncthreads();
  if (warp == 0) {
    const float sum = warp_sum(s_p[0][lane]);
    if (lane == 0) {
      a.term[static_cast<long long>(s) * blocks + eb] = sum;
      if (eb == 0) a.tokens[s] = n;
    }
  }
  __syncthreads();
}

// The whole batch, by one block: terms and tokens of the sequences, squares of
// the segments.
__device__ __forceinline__ void join_batch(const LossArgs& a, int blocks) {
  __shared__ float s_t[32], s_z[32];
  __shared__ int s_m[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float t = 0.0f, z = 0.0f;
  int m = 0;
  bool bad = false;
  for (int i = threadIdx.x; i < a.S * blocks; i += blockDim.x) t += __ldcg(a.term + i);
  for (int i = threadIdx.x; i < a.S; i += blockDim.x) {
    m += __ldcg(a.tokens + i);
    if (a.seq_offsets != nullptr) {
      const int lo = __ldg(a.seq_offsets + i), hi = __ldg(a.seq_offsets + i + 1);
      bad = bad || lo < 0 || hi < lo || hi > a.T;
    }
  }
  if (bad) set_status(a.status, MOE_DEV_BAD_OFFSETS);
  for (int c = threadIdx.x; c < a.chunks; c += blockDim.x) {
    const int t0 = c * a.chunk, t1 = min(t0 + a.chunk, a.T);
    for (int q = sequence_of(a, t0); q < a.S; ++q) {
      int begin, end;
      sequence_span(a, q, &begin, &end);
      if (begin >= t1) break;
      if (max(begin, t0) < min(end, t1)) z += __ldcg(a.seg_z + static_cast<long long>(c) + q);
    }
  }
  t = warp_sum(t);
  z = warp_sum(z);
  m = warp_sum(m);
  if (lane == 0) {
    s_t[warp] = t;
    s_z[warp] = z;
    s_m[warp] = m;
  }
  __syncthreads();
  if (warp == 0) {
    t = warp_sum(s_t[lane]);
    z = warp_sum(s_z[lane]);
    m = warp_sum(s_m[lane]);
    if (lane == 0) {
      const float total = static_cast<float>(m > 0 ? m : 1);
      const float balance = t * (static_cast<float>(a.E) / static_cast<float>(a.k)) / total;
      z /= total;
      a.loss[0] = fmaf(a.balance, balance, a.z * z);
      a.loss[1] = balance;
      a.loss[2] = z;
      a.tokens[a.S] = m;
    }
  }
}

// CLUSTER: the grid is one cluster, which joins its chunks itself.
template <int LANES, int N, int VEC, bool CLUSTER>
__global__ void __launch_bounds__(kFwdThreads) k_loss_chunks(const LossArgs a) {
  __shared__ LossShared sh;
  if constexpr (!CLUSTER) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.done = 0;
  }
  chunk_segments<LANES, N, VEC>(a, blockIdx.x, sh);
  if constexpr (CLUSTER) {
    __shared__ float j_p[32][33];
    __shared__ int j_c[32][33];
    const int blocks = (a.E + 31) / 32;
    cluster_sync();
    for (int i = blockIdx.x; i < a.S * blocks; i += gridDim.x)
      join_sequence(a, i / blocks, i % blocks, blocks, j_p, j_c, sh.n);
    cluster_sync();
    if (blockIdx.x == 0) join_batch(a, blocks);
  }
}

// One block: 32 experts of one sequence.  The last block to end joins the
// sequences.
__global__ void __launch_bounds__(1024) k_loss_join(const LossArgs a) {
  __shared__ float j_p[32][33];
  __shared__ int j_c[32][33];
  __shared__ int j_n[32];
  __shared__ bool s_last;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  join_sequence(a, blockIdx.y, blockIdx.x, gridDim.x, j_p, j_c, j_n);
  if (gridDim.x * gridDim.y > 1) {
    if (threadIdx.x == 0) {
      __threadfence();
      s_last = atomicAdd(a.done, 1u) == gridDim.x * gridDim.y - 1;
      __threadfence();
    }
    __syncthreads();
    if (!s_last) return;
  }
  join_batch(a, gridDim.x);
}

// One group of lanes a token.  f is taken around its mean 1 over the experts,
// which changes nothing in f - <f, p> but keeps the difference of near equals
// exact.  The selected experts' share goes through a row in shared memory, zero
// between tokens: a slot a lane, where slots that name one expert twice are
// added in their order.
template <int LANES, int N, int VEC>
__global__ void __launch_bounds__(kBwdThreads) k_loss_bwd(const LossArgs a) {
  constexpr int kGroups = kBwdThreads / LANES;
  __shared__ __align__(16) float s_row[kGroups][LANES * N];
  const int group = threadIdx.x / LANES, lane = threadIdx.x % LANES;
  const uint32_t mask = group_lanes<LANES>();
  const int t0 = blockIdx.x * a.chunk, t1 = min(t0 + a.chunk, a.T);
  const int total = __ldg(a.tokens + a.S);
  const float scale = (a.dloss != nullptr ? __ldg(a.dloss) : 1.0f) /
                      static_cast<float>(total > 0 ? total : 1);
  float* share = s_row[group];
#pragma unroll
  for (int i = 0; i < N; ++i) share[i * LANES + lane] = 0.0f;
  __syncwarp(mask);
  int have = -1;               // the sequence whose f lies in the registers
  float f[N], next[N];
#pragma unroll
  for (int i = 0; i < N; ++i) f[i] = next[i] = 0.0f;
  if (t0 + group < t1)
    load_row<LANES, N, VEC>(a.logits + static_cast<long long>(t0 + group) * a.E, a.E, lane,
                            -INFINITY, next);
  for (int t = t0 + group; t < t1; t += kGroups) {
    float x[N];
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = next[i];
    if (t + kGroups < t1)
      load_row<LANES, N, VEC>(a.logits + static_cast<long long>(t + kGroups) * a.E, a.E, lane,
                              -INFINITY, next);
    const long long at = static_cast<long long>(t) * a.k;
    float w = 0.0f, dw = 0.0f;
    int idx = -1;
    if (a.dw != nullptr && lane < a.k) {
      w = __ldg(a.topk_w + at + lane);
      dw = __ldg(a.dw + at + lane);
      idx = __ldg(a.topk_idx + at + lane);
    }
    const int s = sequence_of(a, t);
    bool live = s < a.S && (a.mask == nullptr || a.mask[t] != 0);
    if (live && a.seq_offsets != nullptr) live = t >= __ldg(a.seq_offsets + s);
    if (live && s != have) {
      const int n = __ldg(a.tokens + s);
      const float per =
          static_cast<float>(a.E) / (static_cast<float>(a.k) * static_cast<float>(n > 0 ? n : 1));
#pragma unroll
      for (int j = 0; j < N / VEC; ++j)
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          const int e = expert_of<LANES, VEC>(lane, j) + i;
          f[j * VEC + i] =
              e < a.E ? __ldg(a.counts + static_cast<long long>(s) * a.E + e) * per - 1.0f : 0.0f;
        }
      have = s;
    }
    if (live) {
      float inv, dot;
      const float lse = row_softmax<LANES, N, true>(x, inv, f, dot, mask);
      const float b = scale * inv * a.balance;
      const float zz = scale * inv * (2.0f * a.z * lse - a.balance * dot);
#pragma unroll
      for (int i = 0; i < N; ++i) x[i] *= fmaf(b, f[i], zz);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) x[i] = 0.0f;
    }
    if (a.dw != nullptr) {
      float dot = w * dw;
      for (int i = LANES + lane; i < a.k; i += LANES)
        dot = fmaf(__ldg(a.topk_w + at + i), __ldg(a.dw + at + i), dot);
      dot = group_sum<LANES>(dot, mask);
      for (int i0 = 0; i0 < a.k; i0 += LANES) {
        if (i0 > 0) {
          const bool in = i0 + lane < a.k;
          w = in ? __ldg(a.topk_w + at + i0 + lane) : 0.0f;
          dw = in ? __ldg(a.dw + at + i0 + lane) : 0.0f;
          idx = in ? __ldg(a.topk_idx + at + i0 + lane) : -1;
        }
        bool in = i0 + lane < a.k;
        if (in && (idx < 0 || idx >= a.E)) {
          set_status(a.status, MOE_DEV_BAD_EXPERT);
          in = false;
        }
        const float v = w * (dw - dot);
        const uint32_t same = __match_any_sync(mask, in ? idx : -1 - lane);
        // the slots of one expert in their order, one at a time
        for (uint32_t turn = __popc(same & ((1u << (threadIdx.x & 31)) - 1u));
             __any_sync(mask, in); --turn) {
          if (in && turn == 0) {
            share[idx] += v;
            in = false;
          }
          __syncwarp(mask);
        }
      }
#pragma unroll
      for (int j = 0; j < N / VEC; ++j)
#pragma unroll
        for (int i = 0; i < VEC; ++i)
          x[j * VEC + i] += share[expert_of<LANES, VEC>(lane, j) + i];
      __syncwarp(mask);
#pragma unroll
      for (int j = 0; j < N / VEC; ++j)
#pragma unroll
        for (int i = 0; i < VEC; ++i) share[expert_of<LANES, VEC>(lane, j) + i] = 0.0f;
      __syncwarp(mask);
    }
    float* out = a.dlogits + static_cast<long long>(t) * a.E;
#pragma unroll
    for (int j = 0; j < N / VEC; ++j) {
      const int e = expert_of<LANES, VEC>(lane, j);
      if (e >= a.E) continue;
      if constexpr (VEC == 4)
        *reinterpret_cast<float4*>(out + e) =
            make_float4(x[4 * j], x[4 * j + 1], x[4 * j + 2], x[4 * j + 3]);
      else
        out[e] = x[j];
    }
  }
}

// Calls f with the lanes a token, values a lane and vector width for E.
template <typename F>
cudaError_t with_shape(int E, bool vec, F f) {
  if (vec) {
    if (E <= 32) return f.template operator()<8, 4, 4>();
    if (E <= 64) return f.template operator()<8, 8, 4>();
    if (E <= 128) return f.template operator()<32, 4, 4>();
    return f.template operator()<32, 8, 4>();
  }
  if (E <= 8) return f.template operator()<8, 1, 1>();
  if (E <= 32) return f.template operator()<8, 4, 1>();
  if (E <= 64) return f.template operator()<8, 8, 1>();
  if (E <= 128) return f.template operator()<32, 4, 1>();
  return f.template operator()<32, 8, 1>();
}

// Tokens a block takes so that there are about `blocks` of them: 32 to `most`,
// in whole rounds of eight groups.
int chunk_tokens(int T, int blocks, int most) {
  const int want = (T + blocks - 1) / blocks;
  return want <= 32 ? 32 : want >= most ? most : (want + 7) / 8 * 8;
}

// The workspace has to fit whatever GPU the call runs on: for the shortest chunks.
size_t max_segments(const moe_router_loss_desc_t* d) {
  return (static_cast<size_t>(d->T) + 31) / 32 + d->sequences;
}

size_t up16(size_t n) { return (n + 15) / 16 * 16; }

moe_status_t check_loss_desc(const moe_router_loss_desc_t* d) {
  if (!d) return MOE_ERR_NULL;
  if (d->T < 0 || d->T > (1 << 28) || d->E < 1 || d->E > kMaxExperts || d->k < 1 || d->k > d->E ||
      d->k > kMaxTopK || d->sequences < 1 || d->sequences > 65535)
    return MOE_ERR_SHAPE;
  if (!isfinite(d->balance_coef) || !isfinite(d->z_coef)) return MOE_ERR_SHAPE;
  return MOE_OK;
}

bool aligned(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

size_t loss_ws_bytes(const moe_router_loss_desc_t* d) {
  const size_t segs = max_segments(d), blocks = (d->E + 31) / 32;
  return up16(segs * d->E * 4) * 2 + up16(segs * 4) * 2 + up16(d->sequences * blocks * 4) + 16;
}

void fill(LossArgs& a, const moe_router_loss_desc_t* d) {
  a.T = d->T;
  a.E = d->E;
  a.k = d->k;
  a.S = d->sequences;
  a.balance = d->balance_coef;
  a.z = d->z_coef;
}

struct RunChunks {
  const LossArgs& a;
  cudaStream_t s;
  template <int LANES, int N, int VEC>
  cudaError_t operator()() const {
    if (a.chunks > kLossCluster) {
      k_loss_chunks<LANES, N, VEC, false><<<a.chunks, kFwdThreads, 0, s>>>(a);
      return cudaGetLastError();
    }
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = a.chunks;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.chunks);
    cfg.blockDim = dim3(kFwdThreads);
    cfg.stream = s;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k_loss_chunks<LANES, N, VEC, true>, a);
  }
};

struct RunBwd {
  const LossArgs& a;
  cudaStream_t s;
  template <int LANES, int N, int VEC>
  cudaError_t operator()() const {
    k_loss_bwd<LANES, N, VEC><<<a.chunks, kBwdThreads, 0, s>>>(a);
    return cudaGetLastError();
  }
};

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

moe_status_t moe_router_loss_workspace_size(const moe_router_loss_desc_t* desc, size_t* bytes) {
  if (!bytes) return MOE_ERR_NULL;
  const moe_status_t st = check_loss_desc(desc);
  if (st != MOE_OK) return st;
  *bytes = loss_ws_bytes(desc);
  return MOE_OK;
}

moe_status_t moe_router_loss_fwd(const moe_router_loss_desc_t* desc, const float* logits,
                                 const int32_t* topk_idx, const uint8_t* mask,
                                 const int32_t* seq_offsets, int32_t* counts, int32_t* tokens,
                                 float* probs, float* loss, void* ws, size_t ws_bytes,
                                 cudaStream_t stream) {
  moe_status_t st = check_loss_desc(desc);
  if (st != MOE_OK) return st;
  if (!counts || !tokens || !probs || !loss || !ws) return MOE_ERR_NULL;
  if (desc->T > 0 && (!logits || !topk_idx)) return MOE_ERR_NULL;
  if (desc->sequences > 1 && !seq_offsets) return MOE_ERR_NULL;
  if (!aligned(logits, 4) || !aligned(topk_idx, 4) || !aligned(seq_offsets, 4) ||
      !aligned(counts, 4) || !aligned(tokens, 4) || !aligned(probs, 4) || !aligned(loss, 4) ||
      !aligned(ws, 16))
    return MOE_ERR_SHAPE;
  if (ws_bytes < loss_ws_bytes(desc)) return MOE_ERR_WORKSPACE;
  LossArgs a = {};
  int sms;
  st = current_device(&sms, &a.status);
  if (st != MOE_OK) return st;
  fill(a, desc);
  a.logits = logits;
  a.topk_idx = topk_idx;
  a.mask = mask;
  a.seq_offsets = seq_offsets;
  a.counts = counts;
  a.tokens = tokens;
  a.probs = probs;
  a.loss = loss;
  a.chunk = chunk_tokens(a.T, sms, kFwdMostTokens);
  a.chunks = (a.T + a.chunk - 1) / a.chunk;
  const size_t segs = max_segments(desc);
  const int e_blocks = (a.E + 31) / 32;
  char* p = static_cast<char*>(ws);
  auto take = [&p](size_t n) {
    char* q = p;
    p += up16(n);
    return q;
  };
  a.seg_p = reinterpret_cast<float*>(take(segs * a.E * 4));
  a.seg_count = reinterpret_cast<int32_t*>(take(segs * a.E * 4));
  a.seg_z = reinterpret_cast<float*>(take(segs * 4));
  a.seg_tokens = reinterpret_cast<int32_t*>(take(segs * 4));
  a.term = reinterpret_cast<float*>(take(static_cast<size_t>(a.S) * e_blocks * 4));
  a.done = reinterpret_cast<unsigned int*>(take(4));
  // (without tokens one empty chunk, which writes the zeros)
  if (a.chunks == 0) a.chunks = 1;
  if (with_shape(a.E, a.E % 4 == 0 && aligned(logits, 16), RunChunks{a, stream}) != cudaSuccess)
    return MOE_ERR_CUDA;
  if (a.chunks <= kLossCluster) return MOE_OK;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(e_blocks, a.S);
  cfg.blockDim = dim3(1024);
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_loss_join, a) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

moe_status_t moe_router_loss_bwd(const moe_router_loss_desc_t* desc, const float* logits,
                                 const uint8_t* mask, const int32_t* seq_offsets,
                                 const int32_t* counts, const int32_t* tokens, const float* dloss,
                                 const float* dw, const float* topk_w, const int32_t* topk_idx,
                                 float* dlogits, cudaStream_t stream) {
  moe_status_t st = check_loss_desc(desc);
  if (st != MOE_OK) return st;
  if (!counts || !tokens) return MOE_ERR_NULL;
  if (desc->T > 0 && (!logits || !dlogits)) return MOE_ERR_NULL;
  if (dw && (!topk_w || !topk_idx)) return MOE_ERR_NULL;
  if (desc->sequences > 1 && !seq_offsets) return MOE_ERR_NULL;
  if (!aligned(logits, 4) || !aligned(topk_idx, 4) || !aligned(seq_offsets, 4) ||
      !aligned(counts, 4) || !aligned(tokens, 4) || !aligned(dloss, 4) || !aligned(dw, 4) ||
      !aligned(topk_w, 4) || !aligned(dlogits, 4))
    return MOE_ERR_SHAPE;
  LossArgs a = {};
  int sms;
  st = current_device(&sms, &a.status);
  if (st != MOE_OK) return st;
  if (desc->T == 0) return MOE_OK;
  fill(a, desc);
  a.logits = logits;
  a.mask = mask;
  a.seq_offsets = seq_offsets;
  a.counts = const_cast<int32_t*>(counts);
  a.tokens = const_cast<int32_t*>(tokens);
  a.dloss = dloss;
  a.dw = dw;
  a.topk_w = topk_w;
  a.topk_idx = topk_idx;
  a.dlogits = dlogits;
  a.chunk = chunk_tokens(a.T, 8 * sms, 256);
  a.chunks = (a.T + a.chunk - 1) / a.chunk;
  const bool vec = a.E % 4 == 0 && aligned(logits, 16) && aligned(dlogits, 16);
  return with_shape(a.E, vec, RunBwd{a, stream}) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
