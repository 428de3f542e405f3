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
// two kScaleA, kScaleB and 2^x_exp keep them clear of fp16's subnormals.  The
// state X is held in 32 bits, as the fp16 operand and the fp16 of what it
// leaves: a X is exact, and the operand's rounding E enters only through B E,
// which lies in X's own row space -- a direction that X does not have stays
// empty, where a rounded state would fill it and grow by a each step (3.44 by
// default: 485 over five).  In the last two steps B is held as B - s I with
// s = tr(B)/m and X' = (a + s) X + (B - s I) X: near the end B's eigenvalues
// crowd around s, so the rounded part is small.  Not earlier, where E would get
// into the empty directions through s.
//
// The products run on CTA pairs (2-SM MMA), 256 x 256 tiles, as the weight
// gradients of moe_gemm.cu: warp 0 of each CTA feeds a ring of five 32 KB stages
// by TMA, warp 1 of the lead issues the MMAs, eight warps read the accumulators
// of the tile before.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>

#include "moe_internal.h"
#include "moe_ptx.cuh"

namespace moe {
namespace {

constexpr int kTile = 256;                     // both sides of a pair's tile
constexpr int kBK = 64;                        // 64 fp16 = one 128-byte swizzle row
constexpr int kStages = 6;
constexpr int kHalfBytes = 128 * kBK * 2;      // one CTA's half of an operand
constexpr int kStageBytes = 2 * kHalfBytes;
constexpr int kBoxBytes = 64 * kBK * 2;
constexpr int kTmemCols = 2 * kTile;
constexpr int kThreads = 320;
constexpr int kEpiWarps = 8;
constexpr int kEpiBarrier = 1;
constexpr size_t kSmem = 1024 + static_cast<size_t>(kStages) * kStageBytes;
constexpr int kMaxSide = 16384;
constexpr int kMaxSteps = 16;
constexpr int kNormParts = 64;                 // most blocks that share a matrix in the norm
constexpr float kScaleA = 4096.0f;             // A's entries are at most 4
constexpr float kScaleB = 2048.0f;             // B's at most 16

// kind::f16 with fp16 A and B, fp32 accumulation.
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, bool a_mn, bool b_mn) {
  return (1u << 4) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) |
         (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

enum Product : int {
  kGram = 0,     // A = X X^T (or X^T X), upper tiles, mirrored
  kPoly = 1,     // B = b A + c A A, upper tiles, mirrored
  kUpdate = 2,   // X' = a X + B X (or a X + X B)
  kLast = 3      // the same into the caller's tensor
};

struct OrthoArgs {
  CUtensorMap ta;              // first operand, [batch][.][.]
  CUtensorMap tb;
  int batch, M, N, K;          // output rows and columns, contraction
  __half* out_h;               // A, B or X' (operand), rows ld_h apart
  long long ld_h, plane_h;
  __half* x_lo;                // the state's lower half, in place
  const __half* in_h;          // kPoly: A; kUpdate: X
  float* part;                 // kGram: (sum of A_ii, of A_ij^2) by tile, CTA and warp
  float* shift;                // [batch] the s of B - s I
  int use_shift;
  int m;                       // the small side
  float acc_scale;             // accumulator -> what is stored
  float b, c;                  // kPoly
  float a, to_out;             // kUpdate, kLast: X's coefficient, and what all is scaled by
  // kLast: the caller's tensor
  __nv_bfloat16* out;
  long long ld_out, plane_out;
  int out_vec;                 // rows may be written 8 elements at a time
  int* status;
};

struct TileAt {
  int z, mb, nb;
};

// Tile t: matrix after matrix; symmetric products by columns nb of 1, 2, ...
// tiles mb <= nb.
template <bool SYM>
__device__ __forceinline__ TileAt tile_at(int t, int per, int m_tiles) {
  TileAt w;
  w.z = t / per;
  const int r = t - w.z * per;
  if constexpr (SYM) {
    int nb = static_cast<int>((sqrtf(8.0f * r + 1.0f) - 1.0f) * 0.5f);
    while (nb * (nb + 1) / 2 > r) --nb;
    while ((nb + 1) * (nb + 2) / 2 <= r) ++nb;
    w.nb = nb;
    w.mb = r - nb * (nb + 1) / 2;
  } else {
    w.nb = r / m_tiles;
    w.mb = r - w.nb * m_tiles;
  }
  return w;
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ void store_half16(__half* dst, const float (&v)[16]) {
  uint4* p = reinterpret_cast<uint4*>(dst);
#pragma unroll
  for (int q = 0; q < 2; ++q)
    p[q] = make_uint4(pack_half2(v[8 * q], v[8 * q + 1]), pack_half2(v[8 * q + 2], v[8 * q + 3]),
                      pack_half2(v[8 * q + 4], v[8 * q + 5]),
                      pack_half2(v[8 * q + 6], v[8 * q + 7]));
}

__device__ __forceinline__ void load_half16(const __half* src, float (&v)[16]) {
  const uint4* p = reinterpret_cast<const uint4*>(src);
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const uint4 w = p[q];
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
      v[8 * q + 2 * i] = f.x;
      v[8 * q + 2 * i + 1] = f.y;
    }
  }
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

template <int OP, bool AMN, bool BMN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    k_ortho_gemm(const __grid_constant__ OrthoArgs g) {
  constexpr bool kSym = OP == kGram || OP == kPoly;
  constexpr uint32_t kIdesc = idesc_f16(kTile, kTile, AMN, BMN);
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
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const uint32_t tmem_base = s_tmem_base;
  volatile int* abort_flag = &s_abort;
  const int m_tiles = (g.M + kTile - 1) / kTile, n_tiles = (g.N + kTile - 1) / kTile;
  const int per = kSym ? m_tiles * (m_tiles + 1) / 2 : m_tiles * n_tiles;
  const int total = per * g.batch;
  const int num_kb = (g.K + kBK - 1) / kBK;

  if (warp == 0) {
    // ====================== TMA producer (both CTAs) ======================
    if (lane == 0) {
      tma_prefetch_desc(&g.ta);
      tma_prefetch_desc(&g.tb);
      uint32_t stage = 0, phase = 0;
      bool ok = true;
      for (int t = pair; t < total && ok; t += npairs) {
        const TileAt w = tile_at<kSym>(t, per, m_tiles);
        const int m0 = w.mb * kTile + 128 * static_cast<int>(rank);
        const int n0 = w.nb * kTile + 128 * static_cast<int>(rank);
        for (int kb = 0; kb < num_kb; ++kb) {
          if (!mbar_wait(&empty_bar[stage], phase ^ 1u, g.status, abort_flag)) {
            ok = false;
            break;
          }
          uint8_t* sa = smem + stage * kStageBytes;
          uint8_t* sb = sa + kHalfBytes;
          const uint32_t fb = mapa_shared(smem_u32(&full_bar[stage]), 0);
          // boxes past a tensor's end are filled with zeros and count whole
          if (rank == 0) mbar_arrive_expect_tx(&full_bar[stage], 2 * kStageBytes);
          const int k0 = kb * kBK;
          if constexpr (AMN) {
            tma_load_3d_pair(sa, &g.ta, fb, m0, k0, w.z);
            tma_load_3d_pair(sa + kBoxBytes, &g.ta, fb, m0 + 64, k0, w.z);
          } else {
            tma_load_3d_pair(sa, &g.ta, fb, k0, m0, w.z);
          }
          if constexpr (BMN) {
            tma_load_3d_pair(sb, &g.tb, fb, n0, k0, w.z);
            tma_load_3d_pair(sb + kBoxBytes, &g.tb, fb, n0 + 64, k0, w.z);
          } else {
            tma_load_3d_pair(sb, &g.tb, fb, k0, n0, w.z);
          }
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
    }
  } else if (warp == 1) {
    // ====================== MMA issuer (lead CTA only) ====================
    if (lane == 0 && rank == 0) {
      uint32_t stage = 0, phase = 0;
      int it = 0;
      bool ok = true;
      for (int t = pair; t < total && ok; t += npairs, ++it) {
        const int acc = it & 1;
        const uint32_t acc_par = (it >> 1) & 1;
        if (!mbar_wait(&tempty_bar[acc], acc_par ^ 1u, g.status, abort_flag)) break;
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + acc * kTile;
        for (int kb = 0; kb < num_kb; ++kb) {
          if (!mbar_wait(&full_bar[stage], phase, g.status, abort_flag)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t a_base = smem_u32(smem + stage * kStageBytes);
          const uint32_t b_base = a_base + kHalfBytes;
#pragma unroll
          for (int k = 0; k < kBK / 16; ++k) {
            const uint64_t ad = AMN ? sdesc_sw128(a_base + k * 2048, kBoxBytes, 1024)
                                    : sdesc_sw128(a_base + k * 32, 16, 1024);
            const uint64_t bd = BMN ? sdesc_sw128(b_base + k * 2048, kBoxBytes, 1024)
                                    : sdesc_sw128(b_base + k * 32, 16, 1024);
            umma_bf16_pair(d_tmem, ad, bd, kIdesc, (kb > 0 || k > 0) ? 1u : 0u);
          }
          umma_commit_pair(&empty_bar[stage]);
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        umma_commit_pair(&tfull_bar[acc]);
      }
    }
  } else {
    // ====================== epilogue (both CTAs) ==========================
    // eight warps, two per TMEM lane quarter, 16 of every 32 columns each
    const int quarter = warp & 3;
    const int hc = 16 * ((warp - 2) >> 2);
    int it = 0;
    for (int t = pair; t < total; t += npairs, ++it) {
      const TileAt w = tile_at<kSym>(t, per, m_tiles);
      const int row = w.mb * kTile + 128 * static_cast<int>(rank) + quarter * 32 + lane;
      const int n0 = w.nb * kTile + hc;
      const int acc = it & 1;
      const uint32_t acc_par = (it >> 1) & 1;
      const bool mirror = kSym && w.mb != w.nb;
      const bool live = row < g.M;
      float keep = OP == kUpdate || OP == kLast ? g.a : 0.0f;
      float s = 0.0f;
      if constexpr (OP == kUpdate || OP == kLast) {
        if (g.use_shift) keep += __ldcg(g.shift + w.z);
        keep *= g.to_out;
      }
      if constexpr (OP == kPoly) {
        if (g.use_shift && w.mb == w.nb) {
          s = shift_of(g, w.z, per * 2 * kEpiWarps, lane);
          if (w.mb == 0 && rank == 0 && warp == 2 && lane == 0) g.shift[w.z] = s;
        }
      }
      int ok = 1;
      if (lane == 0) ok = mbar_wait(&tfull_bar[acc], acc_par, g.status, abort_flag);
      ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
      if (!ok) break;
      tc_fence_after();
      const uint32_t tbase = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + acc * kTile + hc;
      const int nch = min(kTile / 32, (g.N - n0 + 31) / 32);   // of this warp's columns; may be <= 0
      float tr = 0.0f, sq = 0.0f;
      uint32_t r[16];
#pragma unroll 1
      for (int j = 0; j < nch; ++j) {
        tmem_ld16(tbase + 32 * j, r);
        const int col = n0 + 32 * j;
        float in[16], lo[16], v[16];
        const long long at = static_cast<long long>(w.z) * g.plane_h + row * g.ld_h + col;
        if constexpr (OP != kGram) {
          if (live) load_half16(g.in_h + at, in);
          if constexpr (OP != kPoly) {
            if (live) load_half16(g.x_lo + at, lo);
          }
        }
        tmem_ld_wait16(r);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float x = __uint_as_float(r[i]) * g.acc_scale;
          if constexpr (OP == kGram) {
            v[i] = x;
          } else if constexpr (OP == kPoly) {
            v[i] = fmaf(in[i], g.b * (kScaleB / kScaleA), x);
            if (col + i == row) v[i] -= s * kScaleB;
          } else {
            v[i] = fmaf(keep, in[i] + lo[i], x);
          }
        }
        if constexpr (OP == kGram) {
          // of what is stored, within the matrix
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            v[i] = __half2float(__float2half_rn(v[i]));
            const float x = live && col + i < g.N ? v[i] * (1.0f / kScaleA) : 0.0f;
            sq = fmaf(x, x, sq);
            if (col + i == row) tr += x;
          }
        }
        if (live) {
          if constexpr (kSym) {
            store_half16(g.out_h + at, v);
            if (mirror) {
#pragma unroll
              for (int i = 0; i < 16; ++i)
                if (col + i < g.N)
                  g.out_h[static_cast<long long>(w.z) * g.plane_h + (col + i) * g.ld_h + row] =
                      __float2half_rn(v[i]);
            }
          } else if constexpr (OP == kUpdate) {
            store_half16(g.out_h + at, v);
#pragma unroll
            for (int i = 0; i < 16; ++i) lo[i] = v[i] - __half2float(__float2half_rn(v[i]));
            store_half16(g.x_lo + at, lo);
          } else {
            __nv_bfloat16* dst = g.out + static_cast<long long>(w.z) * g.plane_out +
                                 row * g.ld_out + col;
            if (g.out_vec && col + 16 <= g.N) {
              uint4* p = reinterpret_cast<uint4*>(dst);
#pragma unroll
              for (int q = 0; q < 2; ++q)
                p[q] = make_uint4(pack_bf16x2(v[8 * q], v[8 * q + 1]),
                                  pack_bf16x2(v[8 * q + 2], v[8 * q + 3]),
                                  pack_bf16x2(v[8 * q + 4], v[8 * q + 5]),
                                  pack_bf16x2(v[8 * q + 6], v[8 * q + 7]));
            } else {
#pragma unroll
              for (int i = 0; i < 16; ++i)
                if (col + i < g.N) dst[i] = __float2bfloat16_rn(v[i]);
            }
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(mapa_shared(smem_u32(&tempty_bar[acc]), 0));
      if constexpr (OP == kGram) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
          tr += __shfl_xor_sync(0xFFFFFFFFu, tr, o);
          sq += __shfl_xor_sync(0xFFFFFFFFu, sq, o);
        }
        if (lane == 0)
          reinterpret_cast<float2*>(g.part)[(static_cast<long long>(t) * 2 + rank) * kEpiWarps +
                                            warp - 2] = make_float2(tr, mirror ? 2.0f * sq : sq);
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
struct PrepArgs {
  const void* grad;
  long long ld_g, plane_g;
  const float* mom;            // null: no momentum
  long long ld_m, plane_m;
  float* mom_out;
  long long ld_mo, plane_mo;
  int f32;                     // grad's type
  int vec;                     // rows may be moved 8 elements at a time
  int rows, cols, batch;
  float mu, nu;                // m' = mu m + nu g
  int nesterov;
  double* part;                // [batch][parts]
  int parts;
  float eps, x_scale;          // X is held times x_scale
  __half* x_hi;
  __half* x_lo;
  long long ld_x, plane_x;
};

// U's elements c .. c+n-1 of a row (n <= 8), and where asked the new momentum.
template <bool F32, bool WRITE>
__device__ __forceinline__ void update_of(const PrepArgs& p, int z, int r, int c, int n,
                                          float (&u)[8]) {
  float g[8], m[8];
  const long long at = z * p.plane_g + r * p.ld_g + c;
  if (p.vec) {
    if constexpr (F32) {
      const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p.grad) + at);
      const float4 x = __ldg(q), y = __ldg(q + 1);
      g[0] = x.x, g[1] = x.y, g[2] = x.z, g[3] = x.w;
      g[4] = y.x, g[5] = y.y, g[6] = y.z, g[7] = y.w;
    } else {
      const uint4 x = __ldg(reinterpret_cast<const uint4*>(
          static_cast<const __nv_bfloat16*>(p.grad) + at));
      const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        g[2 * i] = bf16_lo(w[i]);
        g[2 * i + 1] = bf16_hi(w[i]);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if constexpr (F32)
        g[i] = i < n ? __ldg(static_cast<const float*>(p.grad) + at + i) : 0.0f;
      else
        g[i] = i < n ? __bfloat162float(static_cast<const __nv_bfloat16*>(p.grad)[at + i]) : 0.0f;
    }
  }
  if (p.mom == nullptr) {
#pragma unroll
    for (int i = 0; i < 8; ++i) u[i] = g[i];
    return;
  }
  // WRITE: m' from m; otherwise m' as it was written
  const float* src = WRITE ? p.mom : p.mom_out;
  const long long am = WRITE ? z * p.plane_m + r * p.ld_m + c : z * p.plane_mo + r * p.ld_mo + c;
  if (p.vec) {
    const float4* q = reinterpret_cast<const float4*>(src + am);
    const float4 x = q[0], y = q[1];
    m[0] = x.x, m[1] = x.y, m[2] = x.z, m[3] = x.w;
    m[4] = y.x, m[5] = y.y, m[6] = y.z, m[7] = y.w;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) m[i] = i < n ? src[am + i] : 0.0f;
  }
  if constexpr (WRITE) {
#pragma unroll
    for (int i = 0; i < 8; ++i) m[i] = fmaf(p.mu, m[i], p.nu * g[i]);
    float* dst = p.mom_out + z * p.plane_mo + r * p.ld_mo + c;
    if (p.vec) {
      reinterpret_cast<float4*>(dst)[0] = make_float4(m[0], m[1], m[2], m[3]);
      reinterpret_cast<float4*>(dst)[1] = make_float4(m[4], m[5], m[6], m[7]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < n) dst[i] = m[i];
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) u[i] = p.nesterov ? fmaf(p.mu, m[i], p.nu * g[i]) : m[i];
}

// The new momentum, and the squares of U: eight in fp32, the rest in fp64, and
// those eight in fp64 too where their sum leaves fp32's middle range.
template <bool F32>
__global__ void __launch_bounds__(256) k_ortho_norm(const PrepArgs p) {
  __shared__ double s_sum[8];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int z = blockIdx.y;
  const int units = (p.cols + 7) / 8;
  const long long count = static_cast<long long>(p.rows) * units;
  double sum = 0.0;
  for (long long i = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x; i < count;
       i += static_cast<long long>(gridDim.x) * 256) {
    const int r = static_cast<int>(i / units);
    const int c = static_cast<int>(i - static_cast<long long>(r) * units) * 8;
    float u[8];
    update_of<F32, true>(p, z, r, c, min(8, p.cols - c), u);
    float sq = 0.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k) sq = fmaf(u[k], u[k], sq);
    if (sq > 1e-30f && sq < 1e30f) {
      sum += sq;
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) sum += static_cast<double>(u[k]) * u[k];
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
  if (threadIdx.x % 32 == 0) s_sum[threadIdx.x / 32] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < 8; ++w) sum += s_sum[w];
    p.part[static_cast<long long>(z) * p.parts + blockIdx.x] = sum;
  }
}

// X = U / (|U| + eps) as fp16 and the fp16 of the rest.
template <bool F32>
__global__ void __launch_bounds__(256) k_ortho_start(const PrepArgs p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int z = blockIdx.y;
  double sum = 0.0;
  for (int i = threadIdx.x & 31; i < p.parts; i += 32)
    sum += p.part[static_cast<long long>(z) * p.parts + i];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
  const float mul = static_cast<float>(p.x_scale / (sqrt(sum) + p.eps));
  const int units = (p.cols + 7) / 8;
  const long long count = static_cast<long long>(p.rows) * units;
  for (long long i = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x; i < count;
       i += static_cast<long long>(gridDim.x) * 256) {
    const int r = static_cast<int>(i / units);
    const int c = static_cast<int>(i - static_cast<long long>(r) * units) * 8;
    float u[8];
    update_of<F32, false>(p, z, r, c, min(8, p.cols - c), u);
    float lo[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      u[k] *= mul;
      lo[k] = u[k] - __half2float(__float2half_rn(u[k]));
    }
    const long long at = z * p.plane_x + r * p.ld_x + c;
    *reinterpret_cast<uint4*>(p.x_hi + at) =
        make_uint4(pack_half2(u[0], u[1]), pack_half2(u[2], u[3]), pack_half2(u[4], u[5]),
                   pack_half2(u[6], u[7]));
    *reinterpret_cast<uint4*>(p.x_lo + at) =
        make_uint4(pack_half2(lo[0], lo[1]), pack_half2(lo[2], lo[3]), pack_half2(lo[4], lo[5]),
                   pack_half2(lo[6], lo[7]));
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
  int m;                                   // the small side
  long long ld_x, plane_x, ld_a, plane_a;  // elements
  int parts;                               // kGram's sums of a matrix
  size_t x0, x1, lo, a, b, part, norm, shift, bytes;
};

Layout layout_of(const moe_orthogonalize_desc_t* d) {
  Layout w;
  const size_t n = d->batch;
  w.m = d->rows < d->cols ? d->rows : d->cols;
  w.ld_x = up(d->cols, 16);
  w.plane_x = w.ld_x * d->rows;
  w.ld_a = up(w.m, 16);
  w.plane_a = w.ld_a * w.m;
  const int mt = (w.m + kTile - 1) / kTile;
  w.parts = mt * (mt + 1) / 2 * 2 * kEpiWarps;
  size_t at = 0;
  auto take = [&at](size_t b) {
    const size_t p = at;
    at += up(b, 256);
    return p;
  };
  w.x0 = take(n * w.plane_x * 2);
  w.x1 = take(n * w.plane_x * 2);
  w.lo = take(n * w.plane_x * 2);
  w.a = take(n * w.plane_a * 2);
  w.b = take(n * w.plane_a * 2);
  w.part = take(n * w.parts * 8);
  w.norm = take(n * kNormParts * 8);
  w.shift = take(n * 4);
  w.bytes = at > 0 ? at : 256;
  return w;
}

template <int OP, bool AMN, bool BMN>
cudaError_t launch_product(const OrthoArgs& g, int sms, cudaStream_t s) {
  cudaError_t err = cudaFuncSetAttribute(k_ortho_gemm<OP, AMN, BMN>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(kSmem));
  if (err != cudaSuccess) return err;
  const long long mt = (g.M + kTile - 1) / kTile, nt = (g.N + kTile - 1) / kTile;
  const long long tiles =
      g.batch * (OP == kGram || OP == kPoly ? mt * (mt + 1) / 2 : mt * nt);
  const long long pairs = tiles < sms / 2 ? tiles : sms / 2;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(2 * pairs));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_ortho_gemm<OP, AMN, BMN>, g);
}

bool operand_map(CUtensorMap* map, const void* p, long long cols, long long rows, long long batch,
                 long long ld, long long plane, bool mn) {
  return encode_map_3d(map, p, cols, rows, batch, ld * 2, plane * 2, 64, mn ? 64 : 128,
                       CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_DATA_TYPE_FLOAT16);
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
  __half *x_now = half_at(w.x0), *x_next = half_at(w.x1), *A = half_at(w.a), *B = half_at(w.b);
  float* part = reinterpret_cast<float*>(base + w.part);
  float* shift = reinterpret_cast<float*>(base + w.shift);
  const bool tall = desc->rows > desc->cols;
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
  p.part = reinterpret_cast<double*>(base + w.norm);
  p.eps = desc->eps;
  p.x_scale = x_scale;
  p.x_hi = x_now;
  p.x_lo = half_at(w.lo);
  p.ld_x = w.ld_x;
  p.plane_x = w.plane_x;
  const long long units = static_cast<long long>(desc->rows) * ((desc->cols + 7) / 8);
  const long long most = (units + 255) / 256;
  p.parts = static_cast<int>(most < kNormParts ? most : kNormParts);
  const dim3 norm_grid(p.parts, desc->batch);
  const long long start_blocks = (units + 1023) / 1024;
  const dim3 start_grid(static_cast<unsigned>(start_blocks), desc->batch);
  if (f32) {
    k_ortho_norm<true><<<norm_grid, 256, 0, stream>>>(p);
    k_ortho_start<true><<<start_grid, 256, 0, stream>>>(p);
  } else {
    k_ortho_norm<false><<<norm_grid, 256, 0, stream>>>(p);
    k_ortho_start<false><<<start_grid, 256, 0, stream>>>(p);
  }
  if (cudaGetLastError() != cudaSuccess) return MOE_ERR_CUDA;

  OrthoArgs g = {};
  g.batch = desc->batch;
  g.x_lo = p.x_lo;
  g.part = part;
  g.shift = shift;
  g.m = w.m;
  g.b = desc->b;
  g.c = desc->c;
  g.status = status;
  g.out = static_cast<__nv_bfloat16*>(out.p);
  g.ld_out = out.ld;
  g.plane_out = out.plane;
  g.out_vec = out_vec;
  for (int step = 0; step < desc->steps; ++step) {
    const bool last = step + 1 == desc->steps;
    g.use_shift = step + 2 >= desc->steps;
    // A
    g.M = g.N = w.m;
    g.K = tall ? desc->rows : desc->cols;
    g.out_h = A;
    g.ld_h = w.ld_a;
    g.plane_h = w.plane_a;
    g.acc_scale = kScaleA / (x_scale * x_scale);
    if (!operand_map(&g.ta, x_now, desc->cols, desc->rows, desc->batch, w.ld_x, w.plane_x, tall))
      return MOE_ERR_CUDA;
    g.tb = g.ta;
    cudaError_t err = tall ? launch_product<kGram, true, true>(g, sms, stream)
                           : launch_product<kGram, false, false>(g, sms, stream);
    if (err != cudaSuccess) return MOE_ERR_CUDA;
    // B
    g.K = w.m;
    g.in_h = A;
    g.out_h = B;
    g.acc_scale = desc->c * (kScaleB / (kScaleA * kScaleA));
    if (!operand_map(&g.ta, A, w.m, w.m, desc->batch, w.ld_a, w.plane_a, false))
      return MOE_ERR_CUDA;
    g.tb = g.ta;
    if (launch_product<kPoly, false, false>(g, sms, stream) != cudaSuccess) return MOE_ERR_CUDA;
    // X
    g.M = desc->rows;
    g.N = desc->cols;
    g.K = w.m;
    g.in_h = x_now;
    g.out_h = x_next;
    g.ld_h = w.ld_x;
    g.plane_h = w.plane_x;
    g.a = desc->a;
    g.to_out = last ? desc->scale / x_scale : 1.0f;
    g.acc_scale = g.to_out / kScaleB;
    CUtensorMap bm, xm;
    if (!operand_map(&bm, B, w.m, w.m, desc->batch, w.ld_a, w.plane_a, false) ||
        !operand_map(&xm, x_now, desc->cols, desc->rows, desc->batch, w.ld_x, w.plane_x, !tall))
      return MOE_ERR_CUDA;
    g.ta = tall ? xm : bm;
    g.tb = tall ? bm : xm;
    if (last)
      err = tall ? launch_product<kLast, false, false>(g, sms, stream)
                 : launch_product<kLast, false, true>(g, sms, stream);
    else
      err = tall ? launch_product<kUpdate, false, false>(g, sms, stream)
                 : launch_product<kUpdate, false, true>(g, sms, stream);
    if (err != cudaSuccess) return MOE_ERR_CUDA;
    __half* t = x_now;
    x_now = x_next;
    x_next = t;
  }
  return MOE_OK;
}

}  // extern "C"
