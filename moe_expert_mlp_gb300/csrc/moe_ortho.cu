// Orthogonalised updates (see include/moe.h): momentum, then for each matrix
// X = U / (|U|_F + eps) and steps times
//     A = X X^T,  B = b A + c A^2,  X <- a X + B X
// (with X^T X and X B where there are more rows than columns, so A is always
// the small side).  The three products run on the tensor cores; per step and
// matrix of sides m <= n they need m^2 n + m^3 + 2 m^2 n operations, since A and
// A^2 are symmetric: only tiles on or above the diagonal are computed, the
// others are their mirror images.  Everything else is below that.
//
// Numbers.  The operands of the products are fp16: X is bounded (its singular
// values stay below 2, see the descriptor's checks), so fp16's 11 bits serve,
// where bf16's 8 would leave an error of one to several percent.  The powers of
// two kOrthoScaleA and 2^x_exp keep A and X clear of fp16's subnormals.  The
// state X is held in fp32 beside its operand: a X is exact, and the operand's
// rounding E enters only through B E, which lies in X's own column space -- a
// direction that X does not have stays empty, where a rounded state would fill it
// and grow by a each step (3.44 by default: 485 over five).  In the last two steps
// B is held as B - s I with s = tr(B)/m and X' = (a + s) X + (B - s I) X: near the
// end B's eigenvalues crowd around s, so the rounded part is small.  Not earlier,
// where E would get into the empty directions through s.
//
// All products of all steps are one launch.  Its work is a list of 256 x 256
// tiles: group of matrices by group, step by step, in a step A's tiles of every
// matrix, then B's, then X's, dealt out to the CTA pairs in turn.  A tile waits
// only for its own matrix's tiles of the product before, by a counter: those stand
// earlier in the list, so with every pair resident (a cooperative launch) each wait
// ends, and with a few matrices they are done long before, so that no product ends
// in a wave that is half empty (32 matrices of 7168 x 2048: 15 launches took 15.7
// ms; all matrices a product at a time instead of in groups 16.2, in groups 14.5).
//
// A pair works as the weight gradients of moe_gemm.cu do (2-SM MMA): warp 0 of
// each CTA feeds a ring of stages by TMA, warp 1 of the lead issues the MMAs, eight
// warps read the accumulators of the tile before.  A stage takes 128 of the
// contraction (six stages of 64: the same on long lists, 4 % slower on short ones).
// Long lists are bound by the power limit (16 matrices of 2880 x 2880: 1.35 PFLOP/s
// in the first 6 ms, 1.19 held, at 1.5 of 2.07 GHz) and below it by the operands' way
// from L2, 32 KB an SM for every 512 cycles of MMAs.  Short ones are bound by the
// sequence of products: of a 256 x 512 matrix's 4.4 us a product 0.75 are the loads'
// latency, 0.2 the MMAs, 0.3 their signal, 1 the epilogue, 0.5 until its stores are
// out and 0.7 until another SM has seen their count.
// The epilogue keeps to whole lines where it can: the state lies in blocks of 32
// rows by 16 columns in the order in which a warp's lanes take it (rows 4 KB apart
// took four times the passes through L1).  Measured and not kept: sixteen epilogue
// warps (5 % slower: the tile's stores, not latency, set the epilogue's pace), a
// second producer warp, accumulators fetched a chunk ahead (spills), smaller groups
// (one tile a pair instead of two: 64 of 2048 x 1408 4.8 -> 5.6 ms) and larger ones.
#include <math.h>

#include "moe_ortho.cuh"

namespace moe {
namespace {

constexpr int kTile = 256;                     // both sides of a pair's tile
constexpr int kNarrow = 64;                     // a tile's least width
constexpr int kBK = 64;                        // 64 fp16 = one 128-byte swizzle row
constexpr int kSub = 2;                        // such blocks of the contraction a stage
constexpr int kStages = 3;
constexpr int kHalfBytes = 128 * kBK * 2;      // one CTA's half of an operand's block
constexpr int kStageBytes = 2 * kSub * kHalfBytes;
constexpr int kBoxBytes = 64 * kBK * 2;
constexpr int kTmemCols = 2 * kTile;
constexpr int kThreads = 320;
constexpr int kEpiWarps = 8;
constexpr int kMirrorPitch = 40;               // halves from one mirrored row to the next
constexpr int kOutPitch = 18;                  // the same for 32 x 16 of an unaligned result
constexpr int kMirrorBytes = 16 * kMirrorPitch * 2;   // 16 x 32 of a tile, a warp
constexpr size_t kSmem = 1024 + static_cast<size_t>(kStages) * kStageBytes +
                         kEpiWarps * kMirrorBytes;
constexpr int kMaxSide = 16384;
constexpr int kMaxSteps = 16;
constexpr int kNormParts = 608;                // most blocks that share a matrix in the norm

// kind::f16 with fp16 A and B, fp32 accumulation.
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, bool a_mn, bool b_mn) {
  return (1u << 4) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) |
         (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

enum Product : int {
  kGram = 0,     // A = X X^T (or X^T X), upper tiles, mirrored
  kPoly = 1,     // B = b A + c A A - s I and such (term_of), upper tiles, mirrored
  kUpdate = 2,   // X' = (a + s) X + B X (or X B)
  kLast = 3      // the same into the caller's tensor
};

struct OrthoArgs {
  CUtensorMap x_k[2], x_mn[2]; // both X buffers, 64 x 128 boxes and 64 x 64 boxes
  CUtensorMap mat_map[4], mat_half[4];   // the small matrices, 64 x 128 and 64 x 64 boxes
  __half* x[2];                // [batch][rows][ld_x]
  float* state;                // [batch][blocks of 32 x 16], in place
  __half* mat[4];              // [batch][m][ld_a]: A, B and, with joined, two more
  long long ld_x, plane_x, ld_a, plane_a, plane_s;
  int batch, rows, cols, m;
  int steps;                   // of the list: one less than asked for with joined
  int joined;                  // the first of the list are two steps in one
  int groups;                  // of matrices that go through the steps together
  int sym_w, full_w;           // tiles' widths: of A and B, of X
  int tall;                    // more rows than columns: A = X^T X, X' = X B
  float* part;                 // [batch][tiles of A][2 CTAs][8 warps]: sums of A_ii, A_ij^2
  float* shift;                // [batch] s
  unsigned int* done;          // finished halves of small and of X's tiles (counter_at)
  float a, b, c;
  float x_scale, scale;
  __nv_bfloat16* out;
  long long ld_out, plane_out;
  int out_vec;                 // out's rows may be written 16 elements at a time
  int* status;
};

// One tile of the list: rows mb*256 and on, columns nb*width and on; nr: its number
// among its product's of the matrix; q: the small product's number in the step.
struct Work {
  int op, step, z, mb, nb, nr, q;
};

// The list's shape.
struct Plan {
  int r_tiles, c_tiles;            // of X's rows and columns
  int s_tiles, ratio;              // of A's columns, and how many of them are 256 wide
  int sym, full;                   // tiles of A (and B) and of X
  int per_step, per_matrix, total; // of one matrix in a step and in all, of all matrices
};

__host__ __device__ inline int tiles_of(int n, int width) { return (n + width - 1) / width; }

// Tiles on or right of the diagonal's 256 x 256 blocks.
__host__ __device__ inline int sym_tiles(int m, int width) {
  const int rows = tiles_of(m, kTile), ratio = kTile / width;
  return rows * tiles_of(m, width) - ratio * (rows * (rows - 1) / 2);
}

__device__ __forceinline__ Plan plan_of(const OrthoArgs& g) {
  Plan p;
  p.r_tiles = tiles_of(g.rows, kTile);
  p.c_tiles = tiles_of(g.cols, g.full_w);
  p.s_tiles = tiles_of(g.m, g.sym_w);
  p.ratio = kTile / g.sym_w;
  p.sym = sym_tiles(g.m, g.sym_w);
  p.full = p.r_tiles * p.c_tiles;
  p.per_step = 2 * p.sym + p.full;
  p.per_matrix = g.steps * p.per_step + (g.joined ? 4 * p.sym : 0);
  p.total = g.batch * p.per_matrix;
  return p;
}

// Small products of a step, and of all steps before it.
__device__ __forceinline__ int terms_in(const OrthoArgs& g, int step) {
  return g.joined && step == 0 ? 6 : 2;
}
__device__ __forceinline__ int terms_before(const OrthoArgs& g, int step) {
  return step == 0 ? 0 : 2 * step + (g.joined ? 4 : 0);
}

// Two steps in one (with n >= 2 m the 3 m^2 n of a step's long products are more
// than the 3 m^3 that take their place): from A = X X^T alone
//     B = b A + c A A,  N = 2 a B + B B,  A' = a^2 A + N A,  B' = b A' + c A' A',
//     Q = a (B + B') + B' B,  X <- a^2 X + Q X
// as everything here is a polynomial of A, so that the products commute and are
// symmetric.  Only the first two: there A's rounding costs no more than in two
// steps, later it does (five steps, 256 x 900, full rank: 2e-3 of the result, with
// the second and third joined 8e-3).
struct Term {
  int left, right, dst;        // which small matrices
  int in, in2;                 // added times keep; in2 < 0: none
  float scale, keep;           // dst = scale * left right + keep * (in + in2)
};

__device__ __forceinline__ Term term_of(const OrthoArgs& g, int q) {
  const float square = g.c / (kOrthoScaleA * kOrthoScaleA), linear = g.b / kOrthoScaleA;
  switch (q) {
    case 1: return {0, 0, 1, 0, -1, square, linear};
    case 2: return {1, 1, 2, 1, -1, 1.0f, 2.0f * g.a};
    case 3: return {2, 0, 3, 0, -1, 1.0f, g.a * g.a};
    case 4: return {3, 3, 2, 3, -1, square, linear};
    default: return {2, 1, 0, 1, 2, 1.0f, g.a};
  }
}

// The small matrix that X is multiplied by.
__device__ __forceinline__ int factor_of(const OrthoArgs& g, int step) {
  return g.joined && step == 0 ? 0 : 1;
}

// Symmetric products go row by row of 256; X with the small side inside, so that
// the long side's panel is shared by its neighbours.
__device__ __forceinline__ Work work_at(const OrthoArgs& g, const Plan& p, int t) {
  Work w;
  // group i holds the matrices floor(i batch / groups) and on
  const int i = static_cast<int>(
      (static_cast<long long>(t / p.per_matrix + 1) * g.groups - 1) / g.batch);
  const int z0 = static_cast<int>(static_cast<long long>(i) * g.batch / g.groups);
  const int z1 = static_cast<int>(static_cast<long long>(i + 1) * g.batch / g.groups);
  int r = t - z0 * p.per_matrix;
  const int first = (z1 - z0) * (p.per_step + (g.joined ? 4 * p.sym : 0));
  w.step = 0;
  if (r >= first) {
    r -= first;
    const int per_step = (z1 - z0) * p.per_step;
    w.step = 1 + r / per_step;
    r -= (w.step - 1) * per_step;
  }
  const int sym = (z1 - z0) * p.sym, small = terms_in(g, w.step) * sym;
  w.q = 0;
  if (r < small) {
    w.q = r / sym;
    w.op = w.q == 0 ? kGram : kPoly;
    r -= w.q * sym;
    const int z = r / p.sym;
    w.z = z0 + z;
    r -= z * p.sym;
    w.nr = r;
    w.mb = 0;
    for (int n = p.s_tiles; r >= n; n -= p.ratio) {
      r -= n;
      ++w.mb;
    }
    w.nb = w.mb * p.ratio + r;
  } else {
    w.op = w.step + 1 == g.steps ? kLast : kUpdate;
    r -= small;
    const int z = r / p.full;
    w.z = z0 + z;
    r -= z * p.full;
    w.nr = r;
    const int inside = g.tall ? p.c_tiles : p.r_tiles;
    const int outside = r / inside;
    r -= outside * inside;
    w.mb = g.tall ? outside : r;
    w.nb = g.tall ? r : outside;
  }
  return w;
}

// Stages of the contraction, the tile's first column, the columns that its MMAs
// compute (a multiple of 32, or of 128 where the second operand lies along its
// rows), and the operands' ways to lie.
struct Shape {
  int num_st, col0, n_eff;
  bool a_mn, b_mn;
};

__device__ __forceinline__ Shape shape_of(const OrthoArgs& g, const Work& w) {
  Shape s;
  const bool gram = w.op == kGram, update = w.op >= kUpdate;
  s.a_mn = gram && g.tall;
  s.b_mn = (gram && g.tall) || (update && !g.tall);
  const int K = gram ? (g.tall ? g.rows : g.cols) : g.m;
  s.num_st = (K + kSub * kBK - 1) / (kSub * kBK);
  const int width = update ? g.full_w : g.sym_w;
  s.col0 = w.nb * width;
  const int left = (update ? g.cols : g.m) - s.col0;
  const int unit = s.b_mn ? 128 : 32;
  s.n_eff = min(width, (left + unit - 1) / unit * unit);
  return s;
}

// Where matrix z has its two counts, of small and of X's tiles: a line each, as
// every SM asks for them.
__host__ __device__ inline int counter_at(int z, int which) { return 64 * z + 32 * which; }

// Waits until the tiles that w reads are finished; false when that takes too long
// or the CTA has given up.
__device__ __forceinline__ bool wait_inputs(const OrthoArgs& g, const Plan& p, const Work& w,
                                            volatile int* abort_flag) {
  if (w.op == kGram && w.step == 0) return true;
  const bool gram = w.op == kGram;
  const unsigned int* ctr = g.done + counter_at(w.z, gram ? 1 : 0);
  // a matrix's small products follow one another, so their tiles' count tells which
  // of them are finished
  const int before = terms_before(g, w.step) + (w.op == kPoly ? w.q : terms_in(g, w.step));
  // (each of a tile's two CTAs counts)
  const unsigned int target = 2 * (gram ? w.step * p.full : before * p.sym);
  unsigned int v;
  asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(ctr) : "memory");
  if (v >= target) return true;
  const unsigned long long t0 = global_ns();
  while (true) {
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(ctr) : "memory");
    if (v >= target) return true;
    if (*abort_flag) return false;
    if (global_ns() - t0 > kWaitLimitNs) {
      *abort_flag = 1;
      set_status(g.status, MOE_DEV_TIMEOUT);
      return false;
    }
  }
}

// Whether any thread of the epilogue's warps says so; all of them wait here.
__device__ __forceinline__ bool any_of_epilogue(bool p) {
  uint32_t any;
  __syncwarp();
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "bar.red.or.pred q, 1, %2, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(any)
      : "r"(p ? 1u : 0u), "n"(32 * kEpiWarps)
      : "memory");
  return any != 0;
}

// Where the state has the first 8 of row r's 16 elements from column c (a
// multiple of 16) on; the other 8 are 256 further.
__host__ __device__ inline long long state_at(int col_blocks, int r, int c) {
  return (static_cast<long long>(r / 32) * col_blocks + c / 16) * 512 + (r % 32) * 8;
}

// 32 bytes, past L1 (other SMs write them in the same launch).
__device__ __forceinline__ void load_words(const void* p, uint32_t* w) {
  asm volatile("ld.global.cg.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]),
                 "=r"(w[6]), "=r"(w[7])
               : "l"(p));
}

__device__ __forceinline__ void store_words(void* p, const uint32_t (&w)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]),
               "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// s of matrix z from kGram's sums, by one warp: tr(B) / m = (b tr(A) + c |A|^2) / m.
__device__ __forceinline__ float shift_of(const OrthoArgs& g, int z, int parts, int lane) {
  const float2* p = reinterpret_cast<const float2*>(g.part) + static_cast<long long>(z) * parts;
  float tr = 0.0f, sq = 0.0f;
  for (int i = lane; i < parts; i += 32) {
    const float2 v = __ldcg(p + i);
    tr += v.x;
    sq += v.y;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    tr += __shfl_xor_sync(0xFFFFFFFFu, tr, o);
    sq += __shfl_xor_sync(0xFFFFFFFFu, sq, o);
  }
  return (g.b * tr + g.c * sq) / static_cast<float>(g.m);
}

// A pair of fp16 as two fp32 in one operand of the packed arithmetic.
__device__ __forceinline__ F2 half_pair(uint32_t w) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
  return f2(f.x, f.y);
}

__device__ __forceinline__ uint32_t pack_half(F2 v) {
  const float2 f = parts(v);
  return pack_half2(f.x, f.y);
}

// One warp's share of a tile: 32 rows, 16 of every 32 columns.  The loads of the
// state (or of A) run kAhead chunks ahead, the first ones before `ready` waits for
// the accumulator; `read` is called once the accumulator has been read.
constexpr int kAhead = 4;

template <int OP, typename READY, typename READ>
__device__ __forceinline__ bool epilogue(const OrthoArgs& g, const Plan& p, const Work& w,
                                         int width, uint32_t tbase, int row0, int col0, int lane,
                                         int ewarp, uint32_t rank, __half* mirror_buf, READY ready,
                                         READ read) {
  constexpr bool kSym = OP == kGram || OP == kPoly;
  constexpr bool kState = OP == kUpdate || OP == kLast;
  const int M = kSym ? g.m : g.rows, N = kSym ? g.m : g.cols;
  const int row = row0 + lane;
  const bool live = row < M;
  const bool diagonal = kSym && w.nb / p.ratio == w.mb;
  const bool mirror = kSym && !diagonal;
  const bool shifted = w.step + 2 >= g.steps;
  const int nch = min(width / 32, (N - col0 + 31) / 32);   // may be <= 0
  const long long ld = kSym ? g.ld_a : g.ld_x;
  const long long at0 = static_cast<long long>(w.z) * (kSym ? g.plane_a : g.plane_x) + row * ld +
                        col0;
  // v = keep * (what was loaded) + accumulator, where not kGram, and * scale
  Term term = {};
  if constexpr (OP == kPoly) term = term_of(g, w.q);
  float s = 0.0f, keep = 0.0f, scale = 1.0f;
  if constexpr (OP == kGram) {
    scale = kOrthoScaleA / (g.x_scale * g.x_scale);
  } else if constexpr (OP == kPoly) {
    scale = term.scale;
    keep = term.keep;
    if (shifted && diagonal) {
      s = shift_of(g, w.z, p.sym * 2 * kEpiWarps, lane);
      if (w.nr == 0 && rank == 0 && ewarp == 0 && lane == 0) g.shift[w.z] = s;
    }
  } else {
    keep = (g.joined && w.step == 0 ? g.a * g.a : g.a) +
           (shifted ? __ldcg(g.shift + w.z) : 0.0f);
    if constexpr (OP == kLast) scale = g.scale / g.x_scale;
  }
  const F2 keep2 = f2(keep), scale2 = f2(scale);
  const __half* src = g.mat[term.in];
  const __half* src2 = term.in2 > 0 ? g.mat[term.in2] : nullptr;
  __half* dst = OP == kGram ? g.mat[0] : OP == kPoly ? g.mat[term.dst] : g.x[(w.step + 1) & 1];
  constexpr int kBuf = OP == kGram ? 1 : kAhead;
  // kPoly: one or two matrices' fp16; the state's fp32
  uint32_t in[kBuf][OP == kGram ? 8 : 16] = {};
  float* state = nullptr;
  if constexpr (kState)
    state = g.state + w.z * g.plane_s + state_at((N + 15) / 16, row, col0);
  float tr = 0.0f, sq = 0.0f;

  auto fetch = [&](int j, int b) {
    if constexpr (OP != kGram) {
      if (live && j < nch) {
        if constexpr (kState) {
          load_words(state + 1024 * j, &in[b][0]);
          load_words(state + 1024 * j + 256, &in[b][8]);
        } else {
          load_words(src + at0 + 32 * j, &in[b][0]);
          if (src2 != nullptr) load_words(src2 + at0 + 32 * j, &in[b][8]);
        }
      }
    }
  };
  auto chunk = [&](int j, int b) {
    const int col = col0 + 32 * j;
    uint32_t acc[16];
    tmem_ld16(tbase + 32 * j, acc);
    tmem_ld_wait16(acc);
    if (j + 1 == nch) read();
    F2 v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[i] = f2(__uint_as_float(acc[2 * i]), __uint_as_float(acc[2 * i + 1]));
      if constexpr (OP == kPoly) {
        v[i] = fma2(keep2, half_pair(in[b][i]), v[i] * scale2);
        if (src2 != nullptr) v[i] = fma2(keep2, half_pair(in[b][8 + i]), v[i]);
      }
      if constexpr (kState)
        v[i] = fma2(keep2, f2(__uint_as_float(in[b][2 * i]), __uint_as_float(in[b][2 * i + 1])),
                    v[i]);
      if constexpr (OP == kGram || OP == kLast) v[i] = v[i] * scale2;
    }
    if constexpr (OP == kPoly) {
      if (s != 0.0f) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float2 f = parts(v[i]);
          v[i] = f2(col + 2 * i == row ? f.x - s : f.x, col + 2 * i + 1 == row ? f.y - s : f.y);
        }
      }
    }
    fetch(j + kBuf, b);
    uint32_t h[8];
    if constexpr (OP != kLast) {
#pragma unroll
      for (int i = 0; i < 8; ++i) h[i] = pack_half(v[i]);
      if (live) store_words(dst + at0 + 32 * j, h);
    }
    if constexpr (OP == kGram) {
      if (shifted) {             // of what is stored, within the matrix
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float2 q = parts(half_pair(h[i]));
          const float x = live && col + 2 * i < N ? q.x * (1.0f / kOrthoScaleA) : 0.0f;
          const float y = live && col + 2 * i + 1 < N ? q.y * (1.0f / kOrthoScaleA) : 0.0f;
          sq = fmaf(x, x, fmaf(y, y, sq));
          if (col + 2 * i == row) tr += x;
          if (col + 2 * i + 1 == row) tr += y;
        }
      }
    }
    if constexpr (OP == kUpdate) {
      if (live) {
        float x[16];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float2 f = parts(v[i]);
          x[2 * i] = f.x;
          x[2 * i + 1] = f.y;
        }
        store32(state + 1024 * j, reinterpret_cast<const float(&)[8]>(x[0]));
        store32(state + 1024 * j + 256, reinterpret_cast<const float(&)[8]>(x[8]));
      }
    }
    if constexpr (kSym) {
      if (mirror) {              // 16 columns of 32 rows become 16 rows of 32
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const __half2 two = *reinterpret_cast<const __half2*>(&h[i]);
          mirror_buf[(2 * i) * kMirrorPitch + lane] = __low2half(two);
          mirror_buf[(2 * i + 1) * kMirrorPitch + lane] = __high2half(two);
        }
        __syncwarp();
        const int r = lane >> 1, c = 16 * (lane & 1);
        const uint4* q = reinterpret_cast<const uint4*>(mirror_buf + r * kMirrorPitch + c);
        const uint4 q0 = q[0], q1 = q[1];
        const uint32_t t[8] = {q0.x, q0.y, q0.z, q0.w, q1.x, q1.y, q1.z, q1.w};
        if (col + r < N && row0 + c < M)
          store_words(dst + static_cast<long long>(w.z) * g.plane_a + (col + r) * ld + row0 + c, t);
        __syncwarp();
      }
    }
    if constexpr (OP == kLast) {
      __nv_bfloat16* o = g.out + static_cast<long long>(w.z) * g.plane_out + row0 * g.ld_out + col;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 f = parts(v[i]);
        h[i] = pack_bf16x2(f.x, f.y);
      }
      if (g.out_vec && col - col % 32 + 32 <= N) {
        if (live) store_words(o + lane * g.ld_out, h);
      } else {
        // two rows of 16 at a time: by single elements of 32 rows it took eight
        // times as long
        uint32_t* mine = reinterpret_cast<uint32_t*>(mirror_buf) + lane * (kOutPitch / 2);
#pragma unroll
        for (int i = 0; i < 8; ++i) mine[i] = h[i];
        __syncwarp();
        const int c = lane & 15;
        const uint16_t* from = reinterpret_cast<const uint16_t*>(mirror_buf) + c;
#pragma unroll 4
        for (int r = lane >> 4; r < 32; r += 2)
          if (row0 + r < M && col + c < N)
            reinterpret_cast<uint16_t*>(o)[r * g.ld_out + c] = from[r * kOutPitch];
        __syncwarp();
      }
    }
  };

#pragma unroll
  for (int b = 0; b < kBuf; ++b) fetch(b, b);
  if (!ready()) return false;
  if (nch <= 0) read();
#pragma unroll 1
  for (int j = 0; j < nch; j += kBuf) {
#pragma unroll
    for (int b = 0; b < kBuf; ++b)
      if (j + b < nch) chunk(j + b, b);
  }
  if constexpr (OP == kGram) {
    if (shifted) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        tr += __shfl_xor_sync(0xFFFFFFFFu, tr, o);
        sq += __shfl_xor_sync(0xFFFFFFFFu, sq, o);
      }
      if (lane == 0)
        reinterpret_cast<float2*>(g.part)[((static_cast<long long>(w.z) * p.sym + w.nr) * 2 + rank) *
                                              kEpiWarps + ewarp] =
            make_float2(tr, mirror ? 2.0f * sq : sq);
    }
  }
  return true;
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    k_ortho_steps(const __grid_constant__ OrthoArgs g) {
  extern __shared__ uint8_t dyn_smem[];
  __shared__ __align__(8) uint64_t full_bar[kStages];
  __shared__ __align__(8) uint64_t empty_bar[kStages];
  __shared__ __align__(8) uint64_t tfull_bar[2];
  __shared__ __align__(8) uint64_t tempty_bar[2];
  __shared__ uint32_t s_tmem_base;
  __shared__ int s_abort;

  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dyn_smem) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;
  if (threadIdx.x == 0) {
    s_abort = 0;
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full_bar[s], 1);
      mbar_init(&empty_bar[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tfull_bar[a], 1);
      mbar_init(&tempty_bar[a], 2 * kEpiWarps);
    }
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc_pair(&s_tmem_base, kTmemCols);
    tmem_relinquish_pair();
    tc_fence_before();
  }
  __syncthreads();
  cluster_sync();                            // peer barriers initialised before any remote use
  tc_fence_after();
  const uint32_t tmem_base = s_tmem_base;
  volatile int* abort_flag = &s_abort;
  const Plan p = plan_of(g);

  if (warp == 0) {
    // ====================== TMA producer (both CTAs) ======================
    // (the whole warp waits and one elected lane issues: of a single lane's branch
    // each load took 250 cycles to issue and each MMA 95)
    uint32_t stage = 0, phase = 0;
    bool ok = true;
    for (int t = pair; t < p.total && ok; t += npairs) {
      const Work w = work_at(g, p, t);
      const Shape sh = shape_of(g, w);
      const int now = w.step & 1;
      // a CTA's half of the second operand in one or two boxes
      const bool two = sh.n_eff > 128;
      const CUtensorMap *ta, *tb;
      if (w.op == kGram) {
        ta = g.tall ? &g.x_mn[now] : &g.x_k[now];
        tb = g.tall || !two ? &g.x_mn[now] : &g.x_k[now];
      } else if (w.op == kPoly) {
        const Term term = term_of(g, w.q);
        ta = &g.mat_map[term.left];
        tb = two ? &g.mat_map[term.right] : &g.mat_half[term.right];
      } else {
        const int f = factor_of(g, w.step);
        ta = g.tall ? &g.x_k[now] : &g.mat_map[f];
        tb = !g.tall ? &g.x_mn[now] : two ? &g.mat_map[f] : &g.mat_half[f];
      }
      const int m0 = w.mb * kTile + 128 * static_cast<int>(rank);
      const int n0 = sh.col0 + (sh.n_eff / 2) * static_cast<int>(rank);
      const uint32_t tx = 2 * kSub * (kHalfBytes + (two ? kHalfBytes : kBoxBytes));
      ok = __all_sync(0xFFFFFFFFu, wait_inputs(g, p, w, abort_flag));
      // what other SMs stored is now read by TMA: the one proxy fence on the way
      // from their stores, here rather than at each of those
      asm volatile("fence.proxy.async.global;" ::: "memory");
      for (int st = 0; st < sh.num_st && ok; ++st) {
        ok = __all_sync(0xFFFFFFFFu,
                        mbar_wait(&empty_bar[stage], phase ^ 1u, g.status, abort_flag));
        if (!ok) break;
        uint8_t* sa = smem + stage * kStageBytes;
        uint8_t* sb = sa + kSub * kHalfBytes;
        const uint32_t fb = mapa_shared(smem_u32(&full_bar[stage]), 0);
        // boxes past a tensor's end are filled with zeros and count whole
        if (elect_one()) {
          if (rank == 0) mbar_arrive_expect_tx(&full_bar[stage], tx);
#pragma unroll
          for (int u = 0; u < kSub; ++u) {
            const int k0 = (st * kSub + u) * kBK;
            if (sh.a_mn) {
              tma_load_3d_pair(sa + u * kHalfBytes, ta, fb, m0, k0, w.z);
              tma_load_3d_pair(sa + u * kHalfBytes + kBoxBytes, ta, fb, m0 + 64, k0, w.z);
            } else {
              tma_load_3d_pair(sa + u * kHalfBytes, ta, fb, k0, m0, w.z);
            }
            if (sh.b_mn) {
              tma_load_3d_pair(sb + u * kHalfBytes, tb, fb, n0, k0, w.z);
              if (two) tma_load_3d_pair(sb + u * kHalfBytes + kBoxBytes, tb, fb, n0 + 64, k0, w.z);
            } else {
              tma_load_3d_pair(sb + u * kHalfBytes, tb, fb, k0, n0, w.z);
            }
          }
        }
        __syncwarp();
        if (++stage == kStages) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
  } else if (warp == 1) {
    // ====================== MMA issuer (lead CTA only) ====================
    if (rank == 0) {
      uint32_t stage = 0, phase = 0;
      int it = 0;
      bool ok = true;
      for (int t = pair; t < p.total && ok; t += npairs, ++it) {
        const Work w = work_at(g, p, t);
        const Shape sh = shape_of(g, w);
        const uint32_t idesc = idesc_f16(kTile, sh.n_eff, sh.a_mn, sh.b_mn);
        const int acc = it & 1;
        const uint32_t acc_par = (it >> 1) & 1;
        if (!__all_sync(0xFFFFFFFFu,
                        mbar_wait(&tempty_bar[acc], acc_par ^ 1u, g.status, abort_flag)))
          break;
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + acc * kTile;
        for (int st = 0; st < sh.num_st; ++st) {
          ok = __all_sync(0xFFFFFFFFu, mbar_wait(&full_bar[stage], phase, g.status, abort_flag));
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
            const uint32_t a_base = smem_u32(smem + stage * kStageBytes);
            const uint32_t b_base = a_base + kSub * kHalfBytes;
#pragma unroll
            for (int k = 0; k < kSub * kBK / 16; ++k) {
              const uint32_t ab = a_base + (k / 4) * kHalfBytes, bb = b_base + (k / 4) * kHalfBytes;
              const uint64_t ad = sh.a_mn ? sdesc_sw128(ab + k % 4 * 2048, kBoxBytes, 1024)
                                          : sdesc_sw128(ab + k % 4 * 32, 16, 1024);
              const uint64_t bd = sh.b_mn ? sdesc_sw128(bb + k % 4 * 2048, kBoxBytes, 1024)
                                          : sdesc_sw128(bb + k % 4 * 32, 16, 1024);
              umma_bf16_pair(d_tmem, ad, bd, idesc, (st > 0 || k > 0) ? 1u : 0u);
            }
            umma_commit_pair(&empty_bar[stage]);
            if (st + 1 == sh.num_st) umma_commit_pair(&tfull_bar[acc]);
          }
          __syncwarp();
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
      }
    }
  } else {
    // ====================== epilogue (both CTAs) ==========================
    // eight warps, two per TMEM lane quarter, 16 of every 32 columns each
    const int quarter = warp & 3, ewarp = warp - 2;
    const int hc = 16 * (ewarp >> 2);
    __half* mirror_buf = reinterpret_cast<__half*>(smem + kStages * kStageBytes) +
                         ewarp * (kMirrorBytes / 2);
    int it = 0;
    bool failed = false;
    for (int t = pair; t < p.total; t += npairs, ++it) {
      const Work w = work_at(g, p, t);
      const int width = w.op >= kUpdate ? g.full_w : g.sym_w;
      const int row0 = w.mb * kTile + 128 * static_cast<int>(rank) + quarter * 32;
      const int col0 = w.nb * width + hc;
      const int acc = it & 1;
      const uint32_t acc_par = (it >> 1) & 1;
      const uint32_t tbase =
          tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + acc * kTile + hc;
      // what the epilogue reads beside the accumulator is there
      // (one thread asks, as one tells below: with each warp at it the counts' own
      // traffic cost 12 % of 3 matrices of 1001 x 1441)
      if (w.op != kGram) {
        if (ewarp == 0 && lane == 0 && !failed) failed = !wait_inputs(g, p, w, abort_flag);
        if (any_of_epilogue(failed)) break;
      }
      auto ready = [&]() {
        int full = 1;
        if (lane == 0) full = mbar_wait(&tfull_bar[acc], acc_par, g.status, abort_flag);
        full = __shfl_sync(0xFFFFFFFFu, full, 0);
        tc_fence_after();
        return full != 0;
      };
      auto read = [&]() {                    // the accumulator is free again
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_relaxed(mapa_shared(smem_u32(&tempty_bar[acc]), 0));
      };
      if (!failed) {
        bool done;
        if (w.op == kGram)
          done = epilogue<kGram>(g, p, w, width, tbase, row0, col0, lane, ewarp, rank, mirror_buf,
                                 ready, read);
        else if (w.op == kPoly)
          done = epilogue<kPoly>(g, p, w, width, tbase, row0, col0, lane, ewarp, rank, mirror_buf,
                                 ready, read);
        else if (w.op == kUpdate)
          done = epilogue<kUpdate>(g, p, w, width, tbase, row0, col0, lane, ewarp, rank, mirror_buf,
                                   ready, read);
        else
          done = epilogue<kLast>(g, p, w, width, tbase, row0, col0, lane, ewarp, rank, mirror_buf,
                                 ready, read);
        failed = !done;
      }
      if (w.op != kLast) {                   // (the readers fence before their TMA)
        if (any_of_epilogue(failed)) break;
        if (ewarp == 0 && lane == 0)
          asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(
                           g.done + counter_at(w.z, w.op == kUpdate ? 1 : 0))
                       : "memory");
      }
    }
  }

  __syncthreads();
  cluster_sync();                            // no remote arrivals after this point
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, kTmemCols);
  }
}

// ------------------------------------------------------------- preparation
// Bound by memory (4 matrices of 7168 x 2048 with a momentum: 96 us for the 587 MB
// of the first, 138 us for the 587 MB of the second).
constexpr int kPrepUnits = 2;

// The new momentum, and the squares of U.
template <bool F32>
__global__ void __launch_bounds__(256, 3) k_ortho_norm(const PrepArgs p) {
  __shared__ double s_sum[8];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int z = blockIdx.y;
  if (blockIdx.x == 0 && threadIdx.x < 2) p.done[counter_at(z, threadIdx.x)] = 0;
  const unsigned units = (p.cols + 7) / 8;
  const unsigned count = p.rows * units;
  const unsigned stride = gridDim.x * 256;
  double sum = 0.0;
  for (unsigned i0 = blockIdx.x * 256 + threadIdx.x; i0 < count; i0 += kPrepUnits * stride) {
    float g[kPrepUnits][8], m[kPrepUnits][8];
    int r[kPrepUnits], c[kPrepUnits];
#pragma unroll
    for (int q = 0; q < kPrepUnits; ++q) {
      const unsigned i = i0 + q * stride;
      r[q] = i / units;
      c[q] = (i - r[q] * units) * 8;
      if (i >= count) {
#pragma unroll
        for (int k = 0; k < 8; ++k) g[q][k] = 0.0f;
        continue;
      }
      load_grad<F32>(p, z, r[q], c[q], min(8, p.cols - c[q]), g[q]);
      if (p.mom != nullptr)
        load_floats(p.mom + z * p.plane_m + r[q] * p.ld_m + c[q], min(8, p.cols - c[q]), p.vec,
                    m[q]);
    }
#pragma unroll
    for (int q = 0; q < kPrepUnits; ++q) {
      if (i0 + q * stride >= count) continue;
      if (p.mom != nullptr) {
        step_momentum(p, z, r[q], c[q], min(8, p.cols - c[q]), g[q], m[q]);
        direction(p, g[q], m[q]);
      }
    }
    sum += squares_of(g);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
  if (threadIdx.x % 32 == 0) s_sum[threadIdx.x / 32] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < 8; ++w) sum += s_sum[w];
    p.part[static_cast<long long>(z) * kNormParts + blockIdx.x] = sum;
  }
}

// X = U / (|U| + eps), as fp32 and fp16.  A warp takes a block of the state, 32 rows
// by 16 columns, a row a lane: whole sectors of the rows, whole lines of the state.
template <bool F32>
__global__ void __launch_bounds__(256, 4) k_ortho_start(const PrepArgs p) {
  __shared__ float2 s_mul;
  const int z = blockIdx.y;
  const int lane = threadIdx.x & 31;
  wait_for_previous();
  if (threadIdx.x < 32) {          // fp64 for one warp only
    double sum = 0.0;
    for (int i = lane; i < p.parts; i += 32)
      sum += p.part[static_cast<long long>(z) * kNormParts + i];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    if (lane == 0) s_mul = norm_factors(sum, p.x_scale, p.eps);
  }
  __syncthreads();
  const float2 mul = s_mul;
  const int col_blocks = (p.cols + 15) / 16;
  const int blocks = (p.rows + 31) / 32 * col_blocks;
  const bool reads_grad = p.mom == nullptr || p.nesterov;
  for (int i = blockIdx.x * 8 + threadIdx.x / 32; i < blocks; i += gridDim.x * 8) {
    const int rb = i / col_blocks;
    const int r = rb * 32 + lane, c0 = (i - rb * col_blocks) * 16;
    if (r >= p.rows) continue;
    float g[2][8], m[2][8];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int c = c0 + 8 * q, n = min(8, p.cols - c);
      if (n <= 0) continue;
      if (reads_grad) load_grad<F32>(p, z, r, c, n, g[q]);
      if (p.mom != nullptr)
        load_floats(p.mom_out + z * p.plane_mo + r * p.ld_mo + c, n, p.vec, m[q]);
    }
    float* state = p.state + z * p.plane_s + state_at(col_blocks, r, c0);
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int c = c0 + 8 * q;
      // (with an odd number of units the last block's second half stays as it is:
      // what comes of it is not stored)
      if (c >= p.cols) continue;
      float u[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) u[k] = reads_grad ? g[q][k] : 0.0f;
      if (p.mom != nullptr) direction(p, u, m[q]);
#pragma unroll
      for (int k = 0; k < 8; ++k) u[k] = u[k] * mul.x * mul.y;
      *reinterpret_cast<uint4*>(p.x_hi + z * p.plane_x + r * p.ld_x + c) =
          make_uint4(pack_half2(u[0], u[1]), pack_half2(u[2], u[3]), pack_half2(u[4], u[5]),
                     pack_half2(u[6], u[7]));
      store32(state + 256 * q, u);
    }
  }
}

// --------------------------------------------------------------- the host's
size_t up(size_t n, size_t to) { return (n + to - 1) / to * to; }

// The singular values start within [0, 1]; p(s) = a s + b s^3 + c s^5 has to
// keep them below 2 (and B's below 16) for the operands to stay within fp16.
bool coefficients_hold(const moe_orthogonalize_desc_t* d) {
  double top = 1.0;
  for (int k = 0; k < d->steps; ++k) {
    const double t = top * top;
    if (fabs(d->b) * t + fabs(d->c) * t * t > 16.0) return false;
    // p is largest in magnitude at the end or where p' = a + 3 b t + 5 c t^2 = 0
    auto p = [&](double s2) {
      return fabs(sqrt(s2) * (d->a + d->b * s2 + static_cast<double>(d->c) * s2 * s2));
    };
    double next = p(t);
    const double q2 = 5.0 * d->c, q1 = 3.0 * d->b, q0 = d->a;
    double roots[2];
    int n = 0;
    if (q2 != 0.0) {
      const double disc = q1 * q1 - 4.0 * q2 * q0;
      if (disc >= 0.0) {
        roots[n++] = (-q1 + sqrt(disc)) / (2.0 * q2);
        roots[n++] = (-q1 - sqrt(disc)) / (2.0 * q2);
      }
    } else if (q1 != 0.0) {
      roots[n++] = -q0 / q1;
    }
    for (int i = 0; i < n; ++i)
      if (roots[i] > 0.0 && roots[i] < t) next = fmax(next, p(roots[i]));
    top = next;
    if (!(top < 2.0)) return false;
  }
  return true;
}

moe_status_t check_ortho_desc(const moe_orthogonalize_desc_t* d) {
  if (!d) return MOE_ERR_NULL;
  if (d->batch < 0 || d->batch > 65535 || d->rows < 1 || d->rows > kMaxSide || d->cols < 1 ||
      d->cols > kMaxSide || d->steps < 1 || d->steps > kMaxSteps)
    return MOE_ERR_SHAPE;
  if (d->grad_dtype != MOE_DTYPE_BF16 && d->grad_dtype != MOE_DTYPE_FP32)
    return MOE_ERR_UNSUPPORTED;
  if (!(d->eps > 0.0f) || !isfinite(d->eps) || !isfinite(d->a) || !isfinite(d->b) ||
      !isfinite(d->c) || !isfinite(d->momentum) || !isfinite(d->dampening) || !isfinite(d->scale))
    return MOE_ERR_SHAPE;
  if (!coefficients_hold(d)) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

struct Layout {
  bool joined;
  int m;                                   // the small side
  long long ld_x, plane_x, ld_a, plane_a, plane_s;  // elements
  int parts;                               // kGram's sums of a matrix
  size_t x0, x1, state, mat[4], part, norm, shift, done, bytes;
};

// Whether the first two steps are taken as one: where that saves products (see
// term_of), and there are tiles enough that products and not their sequence take the
// time.  (32 matrices of 7168 x 2048: 13.9 -> 12.4 ms; 64 of 2048 x 1024: 2.94 ->
// 2.80 ms, both in the state of this step.)
bool joins_steps(const moe_orthogonalize_desc_t* d) {
  const int m = d->rows < d->cols ? d->rows : d->cols, n = d->rows < d->cols ? d->cols : d->rows;
  return d->steps >= 5 && n >= 2 * m &&
         static_cast<long long>(d->batch) * sym_tiles(m, kTile) >= 128;
}

Layout layout_of(const moe_orthogonalize_desc_t* d) {
  Layout w = {};
  const size_t n = d->batch;
  w.m = d->rows < d->cols ? d->rows : d->cols;
  w.ld_x = up(d->cols, 16);
  w.plane_x = w.ld_x * d->rows;
  w.plane_s = static_cast<long long>((d->rows + 31) / 32) * ((d->cols + 15) / 16) * 512;
  w.ld_a = up(w.m, 16);
  w.plane_a = w.ld_a * w.m;
  w.parts = sym_tiles(w.m, kNarrow) * 2 * kEpiWarps;   // for the narrowest tiles
  if (small_ortho(d->rows, d->cols)) {     // all in registers and shared memory
    w.bytes = 256;
    return w;
  }
  size_t at = 0;
  auto take = [&at](size_t b) {
    const size_t p = at;
    at += up(b, 256);
    return p;
  };
  w.x0 = take(n * w.plane_x * 2);
  w.x1 = take(n * w.plane_x * 2);
  w.state = take(n * w.plane_s * 4);
  w.joined = joins_steps(d);
  for (int i = 0; i < 4; ++i) w.mat[i] = i < 2 || w.joined ? take(n * w.plane_a * 2) : w.mat[0];
  w.part = take(n * w.parts * 8);
  w.norm = take(n * kNormParts * 8);
  w.shift = take(n * 4);
  w.done = take(n * 256);
  w.bytes = at > 0 ? at : 256;
  return w;
}

// Boxes of 64 columns and 64 (half) or 128 rows.
bool operand_map(CUtensorMap* map, const void* p, long long cols, long long rows, long long batch,
                 long long ld, long long plane, bool half) {
  return encode_map_3d(map, p, cols, rows, batch, ld * 2, plane * 2, 64, half ? 64 : 128,
                       CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_DATA_TYPE_FLOAT16);
}

// Every pair stays until the list's end and waits for others' tiles: a
// cooperative launch, so that all are resident.
cudaError_t launch_steps(OrthoArgs& g, int sms, cudaStream_t s) {
  cudaError_t err = cudaFuncSetAttribute(k_ortho_steps, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(kSmem));
  if (err != cudaSuccess) return err;
  // narrower tiles as long as they are one for each pair: a product of few tiles
  // takes as long as one of them (8 matrices of 256 x 512, in the state of this step:
  // 149 -> 117 us)
  const int most = sms / 2;
  auto sym = [&](int width) { return static_cast<long long>(g.batch) * sym_tiles(g.m, width); };
  auto full = [&](int width) {
    return static_cast<long long>(g.batch) * tiles_of(g.rows, kTile) * tiles_of(g.cols, width);
  };
  g.sym_w = g.full_w = kTile;
  while (g.sym_w > (g.tall ? 128 : kNarrow) && sym(g.sym_w / 2) <= most) g.sym_w /= 2;
  while (g.full_w > (g.tall ? kNarrow : 128) && full(g.full_w / 2) <= most) g.full_w /= 2;
  const long long tiles = sym(g.sym_w) > full(g.full_w) ? sym(g.sym_w) : full(g.full_w);
  const long long pairs = tiles < most ? tiles : most;
  // together as many matrices as give A's product two tiles a pair: then a
  // product's inputs are done by the time the list comes to it.  (Not for L2: 8
  // matrices of 2048 x 1408 are 248 MB of operands and state, of which 80 bytes an
  // element pass through DRAM in five steps; but half as many, one tile a pair, took
  // 5.6 ms for 64 instead of 4.8, as each wait stands bare then.)
  const int each = sym_tiles(g.m, g.sym_w);
  const long long together = (2 * pairs + each - 1) / each;
  g.groups = static_cast<int>(g.batch > together ? g.batch / together : 1);
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeCooperative;
  attr.val.cooperative = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(2 * pairs));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_ortho_steps, g);
}

struct Tensor {
  const moe_matrices_t& t;
  size_t size;
  // status of a tensor of the descriptor's shape; clears *vec where its rows
  // cannot be moved 8 elements at a time
  moe_status_t check(const moe_orthogonalize_desc_t* d, bool* vec) const {
    if (!t.p) return d->batch > 0 ? MOE_ERR_NULL : MOE_OK;
    const uintptr_t at = reinterpret_cast<uintptr_t>(t.p);
    if (at % size || t.ld < 0 || t.plane < 0 || (d->rows > 1 && t.ld < d->cols) ||
        t.ld > (1ll << 40) || t.plane > (1ll << 46))
      return MOE_ERR_SHAPE;
    const uint64_t whole = 16 / size;
    if (at % 16 || d->cols % 8 || (d->rows > 1 && t.ld % whole) || (d->batch > 1 && t.plane % whole))
      *vec = false;
    return MOE_OK;
  }
};

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

moe_status_t moe_orthogonalize_workspace_size(const moe_orthogonalize_desc_t* desc,
                                              size_t* bytes) {
  if (!bytes) return MOE_ERR_NULL;
  const moe_status_t st = check_ortho_desc(desc);
  if (st != MOE_OK) return st;
  *bytes = layout_of(desc).bytes;
  return MOE_OK;
}

moe_status_t moe_orthogonalize(const moe_orthogonalize_desc_t* desc, moe_matrices_t grad,
                               moe_matrices_t mom, moe_matrices_t mom_out, moe_matrices_t out,
                               void* ws, size_t ws_bytes, cudaStream_t stream) {
  moe_status_t st = check_ortho_desc(desc);
  if (st != MOE_OK) return st;
  const bool has_mom = desc->momentum != 0.0f || mom.p != nullptr || mom_out.p != nullptr;
  const bool f32 = desc->grad_dtype == MOE_DTYPE_FP32;
  bool vec = true, out_vec = true;
  if ((st = Tensor{grad, static_cast<size_t>(f32 ? 4 : 2)}.check(desc, &vec)) != MOE_OK) return st;
  if (has_mom) {
    if ((st = Tensor{mom, 4}.check(desc, &vec)) != MOE_OK) return st;
    if ((st = Tensor{mom_out, 4}.check(desc, &vec)) != MOE_OK) return st;
  }
  if ((st = Tensor{out, 2}.check(desc, &out_vec)) != MOE_OK) return st;
  // a written matrix keeps clear of the next one
  const long long span = static_cast<long long>(desc->rows - 1);
  if (desc->batch > 1 &&
      (out.plane < span * out.ld + desc->cols ||
       (has_mom && mom_out.plane < span * mom_out.ld + desc->cols)))
    return MOE_ERR_SHAPE;
  if (!ws) return MOE_ERR_NULL;
  if (reinterpret_cast<uintptr_t>(ws) % 256) return MOE_ERR_SHAPE;
  const Layout w = layout_of(desc);
  if (ws_bytes < w.bytes) return MOE_ERR_WORKSPACE;
  int sms, *status;
  if ((st = current_device(&sms, &status)) != MOE_OK) return st;
  if (desc->batch == 0) return MOE_OK;

  char* base = static_cast<char*>(ws);
  auto half_at = [base](size_t at) { return reinterpret_cast<__half*>(base + at); };
  __half* x0 = half_at(w.x0);
  // X times a power of two near sqrt(rows cols), so that its entries are about 1
  // where the norm is 1
  const int x_exp = static_cast<int>(
      lround(0.5 * log2(static_cast<double>(desc->rows) * desc->cols)));
  const float x_scale = ldexpf(1.0f, x_exp);

  PrepArgs p = {};
  p.grad = grad.p;
  p.ld_g = grad.ld;
  p.plane_g = grad.plane;
  p.f32 = f32;
  p.vec = vec;
  p.rows = desc->rows;
  p.cols = desc->cols;
  p.batch = desc->batch;
  if (has_mom) {
    p.mom = static_cast<const float*>(mom.p);
    p.ld_m = mom.ld;
    p.plane_m = mom.plane;
    p.mom_out = static_cast<float*>(mom_out.p);
    p.ld_mo = mom_out.ld;
    p.plane_mo = mom_out.plane;
  }
  p.mu = desc->momentum;
  p.nu = 1.0f - desc->dampening;
  p.nesterov = desc->nesterov;
  p.eps = desc->eps;
  p.x_scale = x_scale;
  if (small_ortho(desc->rows, desc->cols)) {
    SmallOrthoArgs small = {p, static_cast<__nv_bfloat16*>(out.p), out.ld, out.plane, out_vec,
                            desc->steps, desc->a, desc->b, desc->c, desc->scale, status};
    return launch_small_ortho(small, sms, stream) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
  }
  p.part = reinterpret_cast<double*>(base + w.norm);
  p.x_hi = x0;
  p.state = reinterpret_cast<float*>(base + w.state);
  p.plane_s = w.plane_s;
  p.ld_x = w.ld_x;
  p.plane_x = w.plane_x;
  p.done = reinterpret_cast<unsigned int*>(base + w.done);
  const long long units = static_cast<long long>(desc->rows) * ((desc->cols + 7) / 8);
  const long long blocks = (units + 256 * kPrepUnits - 1) / (256 * kPrepUnits);
  p.parts = static_cast<int>(blocks < kNormParts ? blocks : kNormParts);
  // blocks a matrix in the second: enough to fill the GPU, few enough that taking
  // the norm's root does not count
  const long long state_blocks = w.plane_s / 512;
  const long long fill = (8ll * sms + desc->batch - 1) / desc->batch;
  const unsigned start_blocks = static_cast<unsigned>(
      (state_blocks + 7) / 8 < fill ? (state_blocks + 7) / 8 : fill);
  const dim3 norm_grid(p.parts, desc->batch), start_grid(start_blocks, desc->batch);
  cudaLaunchAttribute early;       // placed while the first still runs
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = start_grid;
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  if (f32) {
    k_ortho_norm<true><<<norm_grid, 256, 0, stream>>>(p);
    cudaLaunchKernelEx(&cfg, k_ortho_start<true>, p);
  } else {
    k_ortho_norm<false><<<norm_grid, 256, 0, stream>>>(p);
    cudaLaunchKernelEx(&cfg, k_ortho_start<false>, p);
  }
  if (cudaGetLastError() != cudaSuccess) return MOE_ERR_CUDA;

  OrthoArgs g = {};
  __half* x1 = half_at(w.x1);
  if (!operand_map(&g.x_k[0], x0, desc->cols, desc->rows, desc->batch, w.ld_x, w.plane_x, false) ||
      !operand_map(&g.x_k[1], x1, desc->cols, desc->rows, desc->batch, w.ld_x, w.plane_x, false) ||
      !operand_map(&g.x_mn[0], x0, desc->cols, desc->rows, desc->batch, w.ld_x, w.plane_x, true) ||
      !operand_map(&g.x_mn[1], x1, desc->cols, desc->rows, desc->batch, w.ld_x, w.plane_x, true))
    return MOE_ERR_CUDA;
  for (int i = 0; i < 4; ++i) {
    g.mat[i] = half_at(w.mat[i]);
    if (!operand_map(&g.mat_map[i], g.mat[i], w.m, w.m, desc->batch, w.ld_a, w.plane_a, false) ||
        !operand_map(&g.mat_half[i], g.mat[i], w.m, w.m, desc->batch, w.ld_a, w.plane_a, true))
      return MOE_ERR_CUDA;
  }
  g.x[0] = x0;
  g.x[1] = x1;
  g.state = p.state;
  g.plane_s = w.plane_s;
  g.ld_x = w.ld_x;
  g.plane_x = w.plane_x;
  g.ld_a = w.ld_a;
  g.plane_a = w.plane_a;
  g.batch = desc->batch;
  g.rows = desc->rows;
  g.cols = desc->cols;
  g.m = w.m;
  g.joined = w.joined;
  g.steps = desc->steps - (w.joined ? 1 : 0);
  g.tall = desc->rows > desc->cols;
  g.part = reinterpret_cast<float*>(base + w.part);
  g.shift = reinterpret_cast<float*>(base + w.shift);
  g.done = p.done;
  g.a = desc->a;
  g.b = desc->b;
  g.c = desc->c;
  g.x_scale = x_scale;
  g.scale = desc->scale;
  g.out = static_cast<__nv_bfloat16*>(out.p);
  g.ld_out = out.ld;
  g.plane_out = out.plane;
  g.out_vec = out_vec && reinterpret_cast<uintptr_t>(out.p) % 32 == 0 &&
              (desc->rows == 1 || out.ld % 16 == 0) && (desc->batch == 1 || out.plane % 16 == 0);
  g.status = status;
  return launch_steps(g, sms, stream) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
