// The router's losses and their gradient (see include/moe.h for the formulas).
//
// Both passes are one read of the logits: a token's row lies in the registers
// of a group of 8 lanes, whose exchanges give its maximum, its sum of exponentials
// and, in the backward, <f, p>; the next token's row is on its way meanwhile.  Four
// tokens a warp: with a warp a token and 256 experts an exchange of five steps, the
// reciprocal and the loop count for 8 values a lane, not 32 (178 instructions a token
// in the forward, where this takes 100).  What they cannot do without is that read
// (and the backward's write); the arithmetic, one exponential an element, is below it.
//
// Forward: the tokens are cut into chunks of equal length, one block each, and
// a chunk at the ends of sequences into segments.  Chunks and sequences both
// ascend, so the segment of chunk c and sequence s has the number c + s to
// itself.  A block writes its segments' sums of p, counts and squares, and the
// segments of a sequence are added up in ascending order by a second launch, so the
// result does not depend on the order in which blocks ran.  A few tokens are one
// block's, which keeps its sums to itself: one launch.
#include <math.h>

#include "moe_internal.h"
#include "moe_ptx.cuh"

namespace moe {
namespace {

constexpr int kLanes = 8;              // a token's
constexpr int kLossThreads = 256;
constexpr int kAloneThreads = 1024;    // of a block that takes all tokens, up to 64 experts
constexpr int kSlots = 3;              // of a block's ring: rounds in hand and on their way
constexpr int kMostTokens = 1024;      // of a chunk: a group adds 32 up one by one
// Squares are added up of values times this and their mean is multiplied back, so
// that a sum over up to 2^28 tokens does not leave fp32's range before its mean does.
constexpr float kSquareScale = 1.0f / 16384;

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
  float* z_sum;                // [S]
  unsigned int* done;
  int* status;
  int T, E, k, S, chunk, chunks;
  float balance, z;
};

// Element j of a lane's share of a row: VEC consecutive experts at a time.
template <int VEC>
__device__ __forceinline__ int expert_of(int lane, int j) {
  return (j * kLanes + lane) * VEC;
}

// The lanes of the thread's group.
__device__ __forceinline__ uint32_t group_lanes() {
  return ((1u << kLanes) - 1u) << (threadIdx.x % 32 / kLanes * kLanes);
}

__device__ __forceinline__ float group_max(float v, uint32_t mask) {
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(mask, v, o));
  return v;
}

__device__ __forceinline__ float group_sum(float v, uint32_t mask) {
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) v += __shfl_xor_sync(mask, v, o);
  return v;
}

__device__ __forceinline__ float exp2_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float log2_approx(float x) {
  float r;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float rcp_approx(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Softmax of one row over the group's lanes: x becomes exp(x) up to a factor, inv
// the reciprocal of their sum, and with DOT dot is <f, p>.  Returns logsumexp.  In
// powers of two, exp(x) = 2^(x log2(e) - c) with c = top log2(e) as it is rounded:
// the same for the whole row, so that it cancels in p and is added back in
// logsumexp.  That holds while c is rounded by little: a top beyond kFar is taken off
// the logits first (from 2^31 on c's rounding alone would make sums 0 or inf).  A row
// without a logit above -inf has p = 0 and gives 0; maxima pass over NaN, which then
// reaches the sum.
template <int N, bool DOT>
__device__ __forceinline__ float row_softmax(float (&x)[N], float& inv, const float* f, float& dot,
                                             uint32_t mask) {
  constexpr float kLog2E = 1.44269504088896f, kLn2 = 0.693147180559945f;
  constexpr float kFar = 16777216.0f;      // up to it c is off by one at most
  constexpr int kChains = N < 4 ? 1 : 4;   // of maxima and sums, side by side
  float part[kChains], part_dot[kChains];
#pragma unroll
  for (int i = 0; i < kChains; ++i) part[i] = x[i];
#pragma unroll
  for (int i = kChains; i < N; ++i) part[i % kChains] = fmaxf(part[i % kChains], x[i]);
  float top = part[0];
#pragma unroll
  for (int i = 1; i < kChains; ++i) top = fmaxf(top, part[i]);
  top = group_max(top, mask);
  if (top == -INFINITY) top = 0.0f;
  float base = 0.0f;
  if (!(fabsf(top) < kFar)) {      // (or NaN)
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] -= top;
    base = top;
    top = 0.0f;
  }
  const float c = top * kLog2E;
#pragma unroll
  for (int i = 0; i < kChains; ++i) part[i] = part_dot[i] = 0.0f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    x[i] = exp2_approx(fmaf(x[i], kLog2E, -c));
    part[i % kChains] += x[i];
    if constexpr (DOT) part_dot[i % kChains] = fmaf(f[i], x[i], part_dot[i % kChains]);
  }
  float sum = part[0];
  dot = part_dot[0];
#pragma unroll
  for (int i = 1; i < kChains; ++i) {
    sum += part[i];
    dot += part_dot[i];
  }
  sum = group_sum(sum, mask);
  inv = sum == 0.0f ? 0.0f : rcp_approx(sum);
  if constexpr (DOT) dot = group_sum(dot, mask) * inv;
  return sum == 0.0f ? 0.0f : fmaf(c + log2_approx(sum), kLn2, base);
}

// A lane's share of a row in global memory, by single floats.
template <int N>
__device__ __forceinline__ void load_row(const float* row, int E, int lane, float (&x)[N]) {
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const int e = expert_of<1>(lane, j);
    x[j] = e < E ? __ldg(row + e) : -INFINITY;
  }
}

// A block's tokens t0 .. t1 - 1, G a round: whole rows, which lie one after the
// other, come by bulk copies into a ring in shared memory (with rows of a multiple of
// 16 bytes; otherwise the rows are read where they are needed).
template <int G>
struct RowRing {
  const float* src;
  float* slots;                // kSlots rounds
  uint64_t* full;
  int* status;
  volatile int* abort_flag;
  int t0, t1, E, rounds;

  // One thread.
  __device__ __forceinline__ void load(int r) const {
    const int t = t0 + r * G;
    const uint32_t bytes = static_cast<uint32_t>(min(G, t1 - t)) * E * 4;
    uint64_t* bar = full + r % kSlots;
    mbar_arrive_expect_tx(bar, bytes);
    bulk_load(round(r), src + static_cast<long long>(t) * E, bytes, bar);
  }
  // Whole block.
  __device__ __forceinline__ void start() {
    if (threadIdx.x == 0) {
      *abort_flag = 0;
      for (int i = 0; i < kSlots; ++i) mbar_init(full + i, 1);
      fence_mbar_init();
    }
    __syncthreads();
    if (threadIdx.x == 0)
      for (int r = 0; r < min(kSlots, rounds); ++r) load(r);
  }
  // (a wait that runs out sets the status word; what follows is bounded by it)
  __device__ __forceinline__ void wait(int r) const {
    mbar_wait(full + r % kSlots, (r / kSlots) & 1, status, abort_flag);
  }
  __device__ __forceinline__ float* round(int r) const {
    return slots + (r % kSlots) * (G * E);
  }
};

// A lane's share of a row in shared memory, four floats at a time.
template <int N>
__device__ __forceinline__ void load_shared_row(const float* row, int E, int lane, float (&x)[N]) {
#pragma unroll
  for (int j = 0; j < N / 4; ++j) {
    const int e = expert_of<4>(lane, j);
    const float4 v = e < E ? *reinterpret_cast<const float4*>(row + e)
                           : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
    x[4 * j] = v.x;
    x[4 * j + 1] = v.y;
    x[4 * j + 2] = v.z;
    x[4 * j + 3] = v.w;
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

// The same for one token by a whole block: the ends at or before it, counted, so
// that the loads wait for one another once and not at each step of a search.
template <int THREADS>
__device__ __forceinline__ int first_sequence(const LossArgs& a, int t) {
  if (a.seq_offsets == nullptr || a.S > 4 * THREADS) return sequence_of(a, t);
  int n = 0;
  for (int i = 0; i < a.S; i += THREADS) {
    const int at = i + static_cast<int>(threadIdx.x);
    n += __syncthreads_count(at < a.S && __ldg(a.seq_offsets + min(at, a.S - 1) + 1) <= t);
  }
  return n;
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

// What a block sums up with, a value a warp.
template <int THREADS>
struct LossShared {
  static constexpr int kWarps = THREADS / 32;
  float p[kWarps][kMaxExperts];
  int count[kMaxExperts];
  float z[kWarps];
  int n[kWarps];
};

// A block's segments: sums of p, counts, squares and tokens of chunk c.  `done(s,
// p, count, z, n)` gets segment s's, p and count of expert threadIdx.x.
template <int N, int VEC, int THREADS, typename DONE>
__device__ __forceinline__ void chunk_segments(const LossArgs& a, int c, LossShared<THREADS>& sh,
                                               DONE done) {
  constexpr int kGroups = THREADS / kLanes, kWarps = THREADS / 32;
  extern __shared__ __align__(128) float slots[];
  __shared__ __align__(8) uint64_t full[kSlots];
  __shared__ int s_abort;
  const int group = threadIdx.x / kLanes, lane = threadIdx.x % kLanes;
  const int warp = threadIdx.x >> 5;
  const uint32_t mask = group_lanes();
  const int t0 = c * a.chunk, t1 = min(t0 + a.chunk, a.T);
  RowRing<kGroups> ring = {a.logits, slots, full, a.status, &s_abort, t0, t1, a.E,
                  (t1 - t0 + kGroups - 1) / kGroups};
  if constexpr (VEC == 4) ring.start();
  int cur = 0;                   // rounds before it are used up
  auto release = [&]() {
    __syncthreads();
    if (threadIdx.x == 0 && cur + kSlots < ring.rounds) ring.load(cur + kSlots);
    ++cur;
  };
  int from = t0;                 // also of offsets that descend: a round never comes back
  for (int s = first_sequence<THREADS>(a, t0); s < a.S; ++s) {
    int begin, end;
    sequence_span(a, s, &begin, &end);
    if (begin >= t1) break;
    begin = max(begin, from);
    end = min(end, t1);
    if (begin >= end) continue;
    from = end;
    if (threadIdx.x < kMaxExperts) sh.count[threadIdx.x] = 0;
    __syncthreads();
    float acc[N], z = 0.0f;
    int n = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) acc[i] = 0.0f;
    // whether a token counts and, a slot a lane, its experts: a round ahead
    // (as they are loaded: a comparison would wait for them)
    unsigned next_mask = 1;
    int next_e = -1;
    auto fetch = [&](int t) {
      if (t < begin || t >= end) return;
      if (lane < a.k) next_e = __ldg(a.topk_idx + static_cast<long long>(t) * a.k + lane);
      if (a.mask != nullptr) next_mask = __ldg(a.mask + t);
    };
    const int r0 = (begin - t0) / kGroups, r1 = (end - 1 - t0) / kGroups;
    fetch(t0 + r0 * kGroups + group);
    for (int r = r0; r <= r1; ++r) {
      const int t = t0 + r * kGroups + group;
      const bool live = t >= begin && t < end && next_mask != 0;
      const int mine = next_e;
      if (r < r1) fetch(t + kGroups);
      if constexpr (VEC == 4) {
        while (cur < r) {        // rounds between sequences
          ring.wait(cur);
          release();
        }
        ring.wait(r);
      }
      if (live) {
        float x[N], inv, unused;
        if constexpr (VEC == 4)
          load_shared_row(ring.round(r) + group * a.E, a.E, lane, x);
        else
          load_row(a.logits + static_cast<long long>(t) * a.E, a.E, lane, x);
        const float lse = row_softmax<N, false>(x, inv, nullptr, unused, mask);
#pragma unroll
        for (int i = 0; i < N; ++i) acc[i] = fmaf(x[i], inv, acc[i]);
        const float q = lse * kSquareScale;
        z = fmaf(q, q, z);
        ++n;
        for (int i = lane; i < a.k; i += kLanes) {
          const int e = i < kLanes ? mine : __ldg(a.topk_idx + static_cast<long long>(t) * a.k + i);
          if (e < 0 || e >= a.E) set_status(a.status, MOE_DEV_BAD_EXPERT);
          else atomicAdd(&sh.count[e], 1);
        }
      }
      if constexpr (VEC == 4) {
        if (end >= min(t0 + (r + 1) * kGroups, t1)) release();
      }
    }
    __syncwarp();
    // the groups of a warp, then the warps
#pragma unroll
    for (int o = kLanes; o < 32; o <<= 1) {
#pragma unroll
      for (int i = 0; i < N; ++i) acc[i] += __shfl_xor_sync(0xFFFFFFFFu, acc[i], o);
      z += __shfl_xor_sync(0xFFFFFFFFu, z, o);
      n += __shfl_xor_sync(0xFFFFFFFFu, n, o);
    }
    if (threadIdx.x % 32 < kLanes) {
#pragma unroll
      for (int j = 0; j < N / VEC; ++j)
#pragma unroll
        for (int i = 0; i < VEC; ++i) sh.p[warp][expert_of<VEC>(lane, j) + i] = acc[j * VEC + i];
      if (lane == 0) {
        sh.z[warp] = z;
        sh.n[warp] = n;
      }
    }
    __syncthreads();
    if (threadIdx.x < kMaxExperts) {
      float p = 0.0f;
      z = 0.0f;
      n = 0;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        if (threadIdx.x < a.E) p += sh.p[w][threadIdx.x];
        z += sh.z[w];
        n += sh.n[w];
      }
      done(s, p, threadIdx.x < a.E ? sh.count[threadIdx.x] : 0, z, n);
    }
    __syncthreads();
  }
  if constexpr (VEC == 4)        // no copy outlives the block
    for (int r = cur; r < min(cur + kSlots, ring.rounds); ++r) ring.wait(r);
}

// The losses of all sequences, by one thread.
__device__ __forceinline__ void write_losses(const LossArgs& a, float terms, float squares, int n) {
  const float total = static_cast<float>(n > 0 ? n : 1);
  // N_s f P = E / k * count * P
  const float balance = terms * (static_cast<float>(a.E) / static_cast<float>(a.k)) / total;
  const float z = squares / total * (1.0f / (kSquareScale * kSquareScale));
  // (0 times a loss out of range is not 0)
  a.loss[0] = fmaf(a.balance, a.balance != 0.0f ? balance : 0.0f, a.z != 0.0f ? a.z * z : 0.0f);
  a.loss[1] = balance;
  a.loss[2] = z;
  a.tokens[a.S] = n;
}

__device__ __forceinline__ bool ascends(const LossArgs& a, int s) {
  if (a.seq_offsets == nullptr) return true;
  const int lo = __ldg(a.seq_offsets + s), hi = __ldg(a.seq_offsets + s + 1);
  return lo >= 0 && hi >= lo && hi <= a.T;
}

// ALONE: one block takes every token and writes the results.
template <int N, int VEC, bool ALONE, int THREADS>
__global__ void __launch_bounds__(THREADS, THREADS > kLossThreads ? 1 : N <= 8 ? 4 : 2)
    k_loss_chunks(const LossArgs a) {
  __shared__ LossShared<THREADS> sh;
  if constexpr (!ALONE) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.done = 0;
    chunk_segments<N, VEC, THREADS>(a, blockIdx.x, sh, [&](int s, float p, int count, float z, int n) {
      const long long seg = static_cast<long long>(blockIdx.x) + s;
      if (threadIdx.x < a.E) {
        a.seg_p[seg * a.E + threadIdx.x] = p;
        a.seg_count[seg * a.E + threadIdx.x] = count;
      }
      if (threadIdx.x == 0) {
        a.seg_z[seg] = z;
        a.seg_tokens[seg] = n;
      }
    });
  } else {
    __shared__ float s_t[kMaxExperts / 32];
    // an empty sequence's (a segment's results overwrite them)
    bool bad = false;
    for (int i = threadIdx.x; i < a.S * a.E; i += THREADS) {
      a.probs[i] = 0.0f;
      a.counts[i] = 0;
    }
    for (int i = threadIdx.x; i < a.S; i += THREADS) {
      a.tokens[i] = 0;
      bad = bad || !ascends(a, i);
    }
    if (bad) set_status(a.status, MOE_DEV_BAD_OFFSETS);
    __syncthreads();
    float terms = 0.0f, squares = 0.0f;
    int total = 0;
    chunk_segments<N, VEC, THREADS>(a, 0, sh, [&](int s, float p, int count, float z, int n) {
      const float mean = n > 0 ? p / static_cast<float>(n) : 0.0f;
      if (threadIdx.x < a.E) {
        a.probs[s * a.E + threadIdx.x] = mean;
        a.counts[s * a.E + threadIdx.x] = count;
      }
      if (threadIdx.x == 0) a.tokens[s] = n;
      terms = fmaf(static_cast<float>(count), mean, terms);
      squares += z;
      total += n;
    });
    terms = warp_sum(terms);
    if (threadIdx.x % 32 == 0 && threadIdx.x < kMaxExperts) s_t[threadIdx.x / 32] = terms;
    __syncthreads();
    if (threadIdx.x == 0) {
      terms = 0.0f;
#pragma unroll
      for (int w = 0; w < kMaxExperts / 32; ++w) terms += s_t[w];
      write_losses(a, terms, squares, total);
    }
  }
}

// One block: 32 experts of one sequence, its segments over 32 warps.  The last
// block to end joins the sequences.
__global__ void __launch_bounds__(1024) k_loss_join(const LossArgs a) {
  __shared__ float s_p[32][33];
  __shared__ int s_c[32][33];
  __shared__ float s_z[32], s_t[32];
  __shared__ int s_n[32];
  __shared__ bool s_last;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int s = blockIdx.y, e = blockIdx.x * 32 + lane;
  int begin, end;
  sequence_span(a, s, &begin, &end);             // (inputs: not the launch before's)
  const int c0 = begin / a.chunk, c1 = end > begin ? (end - 1) / a.chunk + 1 : c0;
  if (blockIdx.x == 0 && threadIdx.x == 0 && !ascends(a, s))
    set_status(a.status, MOE_DEV_BAD_OFFSETS);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // eight segments a warp on their way at once; tokens and squares: a segment a lane
  constexpr int kAhead = 8;
  float p = 0.0f, z = 0.0f;
  int count = 0, n = 0;
  for (int c = c0 + warp; c < c1; c += 32 * kAhead) {
    float ps[kAhead];
    int cs[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const long long at = (static_cast<long long>(c) + 32 * i + s) * a.E + e;
      const bool in = c + 32 * i < c1 && e < a.E;
      ps[i] = in ? __ldcg(a.seg_p + at) : 0.0f;
      cs[i] = in ? __ldcg(a.seg_count + at) : 0;
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      p += ps[i];
      count += cs[i];
    }
  }
  for (int c = c0 + threadIdx.x; c < c1; c += 1024) {
    n += __ldcg(a.seg_tokens + static_cast<long long>(c) + s);
    z += __ldcg(a.seg_z + static_cast<long long>(c) + s);
  }
  n = warp_sum(n);
  z = warp_sum(z);
  s_p[warp][lane] = p;
  s_c[warp][lane] = count;
  if (lane == 0) {
    s_n[warp] = n;
    s_z[warp] = z;
  }
  __syncthreads();
  // a warp an expert, its lanes the 32 sums
  p = warp_sum(s_p[lane][warp]);
  count = warp_sum(s_c[lane][warp]);
  n = warp_sum(s_n[lane]);
  const float mean = n > 0 ? p / static_cast<float>(n) : 0.0f;
  const int mine = blockIdx.x * 32 + warp;
  if (lane == 0) {
    if (mine < a.E) {
      a.probs[static_cast<long long>(s) * a.E + mine] = mean;
      a.counts[static_cast<long long>(s) * a.E + mine] = count;
    }
    s_t[warp] = mine < a.E ? static_cast<float>(count) * mean : 0.0f;
  }
  __syncthreads();
  const int blocks = gridDim.x * gridDim.y;
  if (warp == 0) {
    const float sum = warp_sum(s_t[lane]);
    z = warp_sum(s_z[lane]);
    if (blocks == 1) {
      if (lane == 0) {
        a.tokens[0] = n;
        write_losses(a, sum, z, n);
      }
    } else if (lane == 0) {
      a.term[static_cast<long long>(s) * gridDim.x + blockIdx.x] = sum;
      if (blockIdx.x == 0) {
        a.tokens[s] = n;
        a.z_sum[s] = z;
      }
      unsigned int before;
      asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;"
                   : "=r"(before)
                   : "l"(a.done)
                   : "memory");
      s_last = before == static_cast<unsigned int>(blocks - 1);
    }
  }
  if (blocks == 1) return;
  __syncthreads();
  if (!s_last) return;
  float t = 0.0f;
  z = 0.0f;
  n = 0;
  for (int i = threadIdx.x; i < blocks; i += 1024) t += __ldcg(a.term + i);
  for (int i = threadIdx.x; i < a.S; i += 1024) {
    n += __ldcg(a.tokens + i);
    z += __ldcg(a.z_sum + i);
  }
  t = warp_sum(t);
  z = warp_sum(z);
  n = warp_sum(n);
  if (lane == 0) {
    s_t[warp] = t;
    s_z[warp] = z;
    s_n[warp] = n;
  }
  __syncthreads();
  if (warp == 0) {
    t = warp_sum(s_t[lane]);
    z = warp_sum(s_z[lane]);
    n = warp_sum(s_n[lane]);
    if (lane == 0) write_losses(a, t, z, n);
  }
}

// One group of lanes a token.  f is taken around its mean 1 over the experts,
// which changes nothing in f - <f, p> but keeps the difference of near equals
// exact.  A row's gradient goes back into its place in shared memory, where the
// selected experts' share is added to it -- a slot a lane; slots that name one
// expert twice one after the other -- and leaves by a bulk copy.
template <int N, int VEC>
__global__ void __launch_bounds__(kLossThreads, N <= 8 ? 4 : 2) k_loss_bwd(const LossArgs a) {
  constexpr int kGroups = kLossThreads / kLanes;
  extern __shared__ __align__(128) float slots[];
  __shared__ __align__(8) uint64_t full[kSlots];
  __shared__ int s_abort;
  const int group = threadIdx.x / kLanes, lane = threadIdx.x % kLanes;
  const uint32_t mask = group_lanes();
  const int t0 = blockIdx.x * a.chunk, t1 = min(t0 + a.chunk, a.T);
  RowRing<kGroups> ring = {a.logits, slots, full, a.status, &s_abort, t0, t1, a.E,
                  (t1 - t0 + kGroups - 1) / kGroups};
  if constexpr (VEC == 4) ring.start();
  const int total = __ldg(a.tokens + a.S);
  const float scale = (a.dloss != nullptr ? __ldg(a.dloss) : 1.0f) /
                      static_cast<float>(total > 0 ? total : 1);
  // the sequence whose f lies in the registers, and its tokens
  int have = first_sequence<kLossThreads>(a, t0), begin = 0, end = 0;
  float f[N];
#pragma unroll
  for (int i = 0; i < N; ++i) f[i] = 0.0f;
  // a token's mask and, a slot a lane, its weights: a round ahead
  float next_w = 0.0f, next_dw = 0.0f;
  int next_idx = -1;
  unsigned next_mask = 1;        // (as it is loaded: a comparison would wait for it)
  auto fetch = [&](int t) {
    if (t < t1 && a.dw != nullptr && lane < a.k) {
      const long long at = static_cast<long long>(t) * a.k + lane;
      next_w = __ldg(a.topk_w + at);
      next_dw = __ldg(a.dw + at);
      next_idx = __ldg(a.topk_idx + at);
    }
    if (t < t1 && a.mask != nullptr) next_mask = __ldg(a.mask + t);
  };
  fetch(t0 + group);
  for (int r = 0; r < ring.rounds; ++r) {
    const int t = t0 + r * kGroups + group;
    const bool here = t < t1, marked = next_mask != 0;
    const long long at = static_cast<long long>(t) * a.k;
    float w = next_w, dw = next_dw;
    int idx = next_idx;
    fetch(t + kGroups);
    if (here && t >= end) {        // on to the token's sequence (to an empty span if it has none)
      if (have < a.S) sequence_span(a, have, &begin, &end);
      if (t >= end) have = sequence_of(a, t);
      const int s = have;
      if (s < a.S) {
        sequence_span(a, s, &begin, &end);
        const int n = __ldg(a.tokens + s);
        const float per =
            static_cast<float>(a.E) / (static_cast<float>(a.k) * static_cast<float>(n > 0 ? n : 1));
        const int32_t* counts = a.counts + static_cast<long long>(s) * a.E;
#pragma unroll
        for (int j = 0; j < N / VEC; ++j) {
          const int e = expert_of<VEC>(lane, j);
          if constexpr (VEC == 4) {
            const int4 c = e < a.E ? __ldg(reinterpret_cast<const int4*>(counts + e))
                                   : make_int4(0, 0, 0, 0);
            f[4 * j] = fmaf(static_cast<float>(c.x), per, -1.0f);
            f[4 * j + 1] = fmaf(static_cast<float>(c.y), per, -1.0f);
            f[4 * j + 2] = fmaf(static_cast<float>(c.z), per, -1.0f);
            f[4 * j + 3] = fmaf(static_cast<float>(c.w), per, -1.0f);
          } else {
            f[j] = e < a.E ? fmaf(static_cast<float>(__ldg(counts + e)), per, -1.0f) : 0.0f;
          }
        }
      } else {
        begin = end = a.T;
      }
    }
    const bool live = here && t >= begin && t < end && marked;
    float* row = slots + group * a.E;
    if constexpr (VEC == 4) {
      ring.wait(r);
      row = ring.round(r) + group * a.E;
    }
    if (here) {
      float x[N];
      if (live) {
        if constexpr (VEC == 4)
          load_shared_row(row, a.E, lane, x);
        else
          load_row(a.logits + static_cast<long long>(t) * a.E, a.E, lane, x);
        float inv, dot;
        const float lse = row_softmax<N, true>(x, inv, f, dot, mask);
        const float b = scale * inv * a.balance;
        const float zz = scale * inv * (2.0f * a.z * lse - a.balance * dot);
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] *= fmaf(b, f[i], zz);
      } else {
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] = 0.0f;
      }
#pragma unroll
      for (int j = 0; j < N / VEC; ++j) {
        const int e = expert_of<VEC>(lane, j);
        if (e >= a.E) continue;
        if constexpr (VEC == 4)
          *reinterpret_cast<float4*>(row + e) =
              make_float4(x[4 * j], x[4 * j + 1], x[4 * j + 2], x[4 * j + 3]);
        else
          row[e] = x[j];
      }
      __syncwarp(mask);
      if (a.dw != nullptr) {
        float dot = w * dw;
        for (int i = kLanes + lane; i < a.k; i += kLanes)
          dot = fmaf(__ldg(a.topk_w + at + i), __ldg(a.dw + at + i), dot);
        dot = group_sum(dot, mask);
        for (int i0 = 0; i0 < a.k; i0 += kLanes) {
          bool in = i0 + lane < a.k;
          if (i0 > 0) {
            w = in ? __ldg(a.topk_w + at + i0 + lane) : 0.0f;
            dw = in ? __ldg(a.dw + at + i0 + lane) : 0.0f;
            idx = in ? __ldg(a.topk_idx + at + i0 + lane) : -1;
          }
          if (in && (idx < 0 || idx >= a.E)) {
            set_status(a.status, MOE_DEV_BAD_EXPERT);
            in = false;
          }
          const float v = w * (dw - dot);
          // slots that name one expert wait for those before them
          const uint32_t same = __match_any_sync(mask, in ? idx : -1 - lane);
          int turn = __popc(same & ((1u << (threadIdx.x & 31)) - 1u));
          if (in && turn == 0) row[idx] += v;
          __syncwarp(mask);
          while (__any_sync(mask, in && turn > 0)) {
            if (in && --turn == 0) row[idx] += v;
            __syncwarp(mask);
          }
        }
      }
      if constexpr (VEC == 1) {
        float* out = a.dlogits + static_cast<long long>(t) * a.E;
        for (int e = lane; e < a.E; e += kLanes) out[e] = row[e];
        __syncwarp(mask);
      }
    }
    if constexpr (VEC == 4) {
      fence_proxy_async_smem();
      __syncthreads();
      if (threadIdx.x == 0) {
        const int first = t0 + r * kGroups;
        bulk_store(a.dlogits + static_cast<long long>(first) * a.E, ring.round(r),
                   static_cast<uint32_t>(min(kGroups, t1 - first)) * a.E * 4);
        bulk_commit();
        // the round before has left its slot, which is the next load's
        bulk_wait_read<1>();
        if (r > 0 && r - 1 + kSlots < ring.rounds) ring.load(r - 1 + kSlots);
      }
    }
  }
  if constexpr (VEC == 4) {
    if (threadIdx.x == 0) bulk_wait_all();
  }
}

// Calls f with the values a lane and the vector width for E.
template <typename F>
cudaError_t with_shape(int E, bool vec, F f) {
  if (vec) {
    if (E <= 32) return f.template operator()<4, 4>();
    if (E <= 64) return f.template operator()<8, 4>();
    if (E <= 128) return f.template operator()<16, 4>();
    return f.template operator()<32, 4>();
  }
  if (E <= 8) return f.template operator()<1, 1>();
  if (E <= 32) return f.template operator()<4, 1>();
  if (E <= 64) return f.template operator()<8, 1>();
  if (E <= 128) return f.template operator()<16, 1>();
  return f.template operator()<32, 1>();
}

// Tokens a block takes so that there are about `blocks` of them, 32 to `most`.
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
  return up16(segs * d->E * 4) * 2 + up16(segs * 4) * 2 + up16(d->sequences * blocks * 4) +
         up16(d->sequences * 4) + 16;
}

void fill(LossArgs& a, const moe_router_loss_desc_t* d) {
  a.T = d->T;
  a.E = d->E;
  a.k = d->k;
  a.S = d->sequences;
  a.balance = d->balance_coef;
  a.z = d->z_coef;
}

// K's rows in shared memory: `slots` rounds of a row of at most N kLanes experts for
// each group.  The limit is the kernel's, not the call's: it is set for the most
// experts that K takes, so that calls at once do not lower it under one another.
template <int N, typename K>
cudaError_t launch_rows(K kernel, const LossArgs& a, int blocks, int threads, int slots,
                        cudaStream_t s) {
  const int column = threads / kLanes * slots * 4, bytes = column * a.E;   // of an expert, of all
  if (bytes > 8 * 1024) {        // with the static part possibly over 48 KB
    const int most = column * (N * kLanes < kMaxExperts ? N * kLanes : kMaxExperts);
    const cudaError_t err =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    if (err != cudaSuccess) return err;
  }
  kernel<<<blocks, threads, bytes, s>>>(a);
  return cudaGetLastError();
}

struct RunChunks {
  const LossArgs& a;
  bool alone;
  cudaStream_t s;
  template <int N, int VEC>
  cudaError_t operator()() const {
    constexpr int kSlotsOf = VEC == 4 ? kSlots : 1;
    if (alone) {
      constexpr int kThreads = N <= 8 ? kAloneThreads : kLossThreads;
      return launch_rows<N>(k_loss_chunks<N, VEC, true, kThreads>, a, 1, kThreads, kSlotsOf, s);
    }
    return launch_rows<N>(k_loss_chunks<N, VEC, false, kLossThreads>, a, a.chunks, kLossThreads,
                          kSlotsOf, s);
  }
};

struct RunBwd {
  const LossArgs& a;
  cudaStream_t s;
  template <int N, int VEC>
  cudaError_t operator()() const {
    return launch_rows<N>(k_loss_bwd<N, VEC>, a, a.chunks, kLossThreads, VEC == 4 ? kSlots : 1, s);
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
  a.chunk = chunk_tokens(a.T, (a.E <= 64 ? 4 : 2) * sms, kMostTokens);
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
  a.z_sum = reinterpret_cast<float*>(take(static_cast<size_t>(a.S) * 4));
  a.done = reinterpret_cast<unsigned int*>(take(4));
  // (with many sequences one block would take them one after the other)
  // four rounds at most
  const bool alone = a.T <= (a.E <= 64 ? kAloneThreads : kLossThreads) / 2 && a.S <= 8;
  if (alone) a.chunk = a.T;
  const bool vec = a.E % 4 == 0 && aligned(logits, 16);
  if (a.chunks > 0 || alone) {
    if (with_shape(a.E, vec, RunChunks{a, alone, stream}) != cudaSuccess) return MOE_ERR_CUDA;
  } else if (cudaMemsetAsync(a.done, 0, 4, stream) != cudaSuccess) {
    return MOE_ERR_CUDA;
  }
  if (alone) return MOE_OK;
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
  a.chunk = chunk_tokens(a.T, (a.E <= 64 ? 4 : 2) * sms, kMostTokens);
  a.chunks = (a.T + a.chunk - 1) / a.chunk;
  const bool vec = a.E % 4 == 0 && aligned(logits, 16) && aligned(dlogits, 16) &&
                   aligned(counts, 16);
  return with_shape(a.E, vec, RunBwd{a, stream}) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
