// Orthogonalised updates of small matrices: a short side of at most 128 and a
// long one that a cluster's registers hold.  One launch, one cluster a matrix.
//
// CTA r of the cluster keeps columns r n_c .. of X (the short side m along the
// rows; a tall matrix is taken transposed) as fp32 in the accumulators of its
// warps, and as the products' fp16 operand in shared memory.  A step is
//     P_r = X_r X_r^T             each CTA, over its own columns
//     A = sum_r P_r               CTA r adds up a share of the rows, in the order
//                                 of the CTAs, and puts them into everyone's A
//     B = b A + c A A - s I       everyone, all of it: m^3 is less than the wait
//     X_r <- (a + s) X_r + B X_r  accumulators scaled, the product added to them
// with no access to global memory between the read of the gradient and the write of
// the result, and no state but registers.  What goes from CTA to CTA is counted by a
// barrier of the CTA that needs it, instead of a barrier of all.  Operands and
// rounding are those of moe_ortho.cu.  These sizes are bound by latency, of such
// exchanges and of chains of small products, which mma.sync starts and ends in tens
// of cycles; a tcgen05 tile would be mostly empty at m = 64 and has to come back
// from TMEM each time (64 x 2048 with a momentum: 15 products of the general kernel
// took 139 us, this 24.6).  A step of it is 6,200 cycles: 900 for the first product and
// 1,000 for the last (the operands' way out of shared memory), 800 for the second,
// 3,300 for the two exchanges.  With sides of 65 to 128 the exchanges are most of a
// step, as shared memory of other CTAs gives and takes some 10 bytes a cycle.
#include <math.h>

#include <atomic>

#include "moe_ortho.cuh"

namespace moe {
namespace {

constexpr int kSmallThreads = 512;
constexpr int kSmallWarps = 16;
constexpr int kPortable = 8;                   // CTAs of a cluster that every GPC holds
constexpr int kMaxCluster = 16;
constexpr int kUnits = 4;                      // of 8 elements that a thread loads at once

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

// c += a b: 16 x 16 by 16 x 8.
__device__ __forceinline__ void mma16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                      uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float4 ld_cluster4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// A part of this CTA's shared memory into another's, counted by a barrier there.
__device__ __forceinline__ void send(uint32_t to, uint32_t from, uint32_t bytes, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, "
      "[%3];" ::"r"(to),
      "r"(from), "r"(bytes), "r"(bar)
      : "memory");
}

// 8 bytes into a CTA of the cluster, counted by a barrier of the same CTA.
__device__ __forceinline__ void st_async2(uint32_t addr, uint32_t lo, uint32_t hi, uint32_t bar) {
  asm volatile(
      "st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v2.b32 [%0], {%1, %2}, [%3];" ::"r"(
          addr),
      "r"(lo), "r"(hi), "r"(bar)
      : "memory");
}

// Waits for what other CTAs send (their stores, so acquired from the cluster).  A
// CTA that gives up goes on with what it has: nothing that it reads decides where it
// reads or writes, or for how long.
__device__ __forceinline__ void wait_sent(uint64_t* bar, uint32_t parity, int* status,
                                          volatile int* abort_flag) {
  const uint32_t at = smem_u32(bar);
  unsigned long long t0 = 0;
  for (unsigned n = 0;; ++n) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(at), "r"(parity)
        : "memory");
    if (ok) return;
    if (n % 32 != 31) continue;
    if (*abort_flag) return;
    const unsigned long long now = global_ns();
    if (t0 == 0) t0 = now;
    if (now - t0 > kWaitLimitNs) {
      *abort_flag = 1;
      set_status(status, MOE_DEV_TIMEOUT);
      return;
    }
  }
}

__device__ __forceinline__ void st_cluster_f64(uint32_t addr, double v) {
  asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(addr), "d"(v) : "memory");
}

// The two halves of cluster_sync(), of all threads.
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// MP: the short side, padded; NB: blocks of 8 columns a warp of X.
template <int MP, int NB>
struct SmallShape {
  static constexpr int kRowWarps = MP / 32;              // 32 rows each
  static constexpr int kColWarps = kSmallWarps / kRowWarps;
  static constexpr int kCols = kColWarps * 8 * NB;       // a CTA's columns
  static constexpr int kPitchX = kCols + 8;              // halves: 16 bytes past whole lines, so
  static constexpr int kPitchA = MP + 8;                 // that 8 rows lie in different banks
  static constexpr int kPitchP = MP + 4;                 // floats
  static constexpr int kPitchU = kCols + 8;              // floats, of the gradient's stage
  static constexpr int kPitchT = MP + 4;                 // the same of a tall matrix: along m
  static constexpr int kPitchY = MP + 8;                 // halves, of a tall result
  static constexpr int kX = MP * kPitchX * 2;
  static constexpr int kA = MP * kPitchA * 2;
  static constexpr int kP = MP * kPitchP * 4;
  static constexpr int kR = (MP + kMaxCluster) * kPitchP * 4;   // a share of rows from each CTA
  // P's rows go to the CTA that adds them up, or that CTA reads them: 17 KB by copies
  // and a barrier that counts them in 2,700 cycles until A is there, read after a
  // barrier of the cluster in 4,000; 66 KB are faster read (32 matrices of 128 x 512:
  // sent 61 us, read 50)
  static constexpr bool kSend = MP == 64;
  static constexpr int kBAt = kX + kA;
  static constexpr int kPAt = kBAt + kA;
  static constexpr int kRAt = kPAt + kP;
  static constexpr int kU = kCols * kPitchT > MP * kPitchU ? kCols * kPitchT * 4 : MP * kPitchU * 4;
  static constexpr int kProducts = kSend ? kRAt + kR : kPAt + kP;
  static constexpr int kBytes = kProducts > kU ? kProducts : kU;
  static_assert(kCols * kPitchY * 2 <= kBytes, "the result goes by way of it");
};

// Rows r0 .. r0+16 MB, columns c0 .. c0+16 NB2 of L L^T's share over k: L in shared
// memory, row-major.
template <int MB, int NB2>
__device__ __forceinline__ void rows_product(float (&acc)[MB][2 * NB2][4], uint32_t base, int pitch,
                                             int r0, int c0, int k, int lane) {
#pragma unroll
  for (int i = 0; i < MB; ++i)
#pragma unroll
    for (int j = 0; j < 2 * NB2; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) acc[i][j][q] = 0.0f;
  const uint32_t a0 = base + ((r0 + lane % 16) * pitch + lane / 16 * 8) * 2;
  const uint32_t b0 = base + ((c0 + lane / 16 * 8 + lane % 8) * pitch + lane / 8 % 2 * 8) * 2;
#pragma unroll(MB == 1 ? 4 : 2)
  for (int k0 = 0; k0 < k; k0 += 16) {
    uint32_t a[MB][4], b[NB2][4];
#pragma unroll
    for (int i = 0; i < MB; ++i) ldsm4(a0 + (16 * i * pitch + k0) * 2, a[i]);
#pragma unroll
    for (int j = 0; j < NB2; ++j) ldsm4(b0 + (16 * j * pitch + k0) * 2, b[j]);
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
      for (int j = 0; j < NB2; ++j) {
        mma16(acc[i][2 * j], a[i], b[j][0], b[j][1]);
        mma16(acc[i][2 * j + 1], a[i], b[j][2], b[j][3]);
      }
  }
}

template <int MP, int NB>
__global__ void __launch_bounds__(kSmallThreads, 1) k_ortho_small(const __grid_constant__ SmallOrthoArgs g) {
  using S = SmallShape<MP, NB>;
  // a warp's block of A and B: 32 x 32 of 128, 16 x 16 of 64
  constexpr int MB = MP / 64, NB2 = MP / 64;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ __align__(8) uint64_t p_bar, a_bar;
  __shared__ double s_norm[kMaxCluster];
  __shared__ double s_part[kSmallThreads];
  __shared__ float s_warp[kSmallWarps];
  __shared__ float2 s_mul;
  __shared__ float s_diag[MP];
  __shared__ volatile int s_abort;
  __half* X = reinterpret_cast<__half*>(smem);
  __half* A = reinterpret_cast<__half*>(smem + S::kX);
  __half* B = reinterpret_cast<__half*>(smem + S::kBAt);
  float* P = reinterpret_cast<float*>(smem + S::kPAt);
  float* U = reinterpret_cast<float*>(smem);
  const PrepArgs& p = g.in;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  uint32_t ctas;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(ctas));
  const int z = blockIdx.x / ctas;
  const bool tall = p.rows > p.cols;
  const int m = tall ? p.cols : p.rows, n = tall ? p.rows : p.cols;
  const int c0 = static_cast<int>(rank) * S::kCols;

  if (threadIdx.x == 0) {
    s_abort = 0;
    mbar_init(&p_bar, 1);
    mbar_init(&a_bar, 1);
    fence_mbar_init();
  }
  __syncthreads();
  cluster_arrive();                          // this CTA has started
  // ---- the gradient and the momentum: this CTA's columns of U, and their squares
  double sum = 0.0;
  float middle = 0.0f;
  bool odd = false;                          // squares that fp32 does not hold
  {
    if (m < MP || c0 + S::kCols > n) {
      for (int i = threadIdx.x; i < S::kU / 16; i += kSmallThreads)
        reinterpret_cast<float4*>(U)[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      __syncthreads();
    }
    // along the caller's rows, 8 at a time: rows of this CTA's part
    const int row0 = tall ? c0 : 0, row1 = tall ? min(c0 + S::kCols, n) : m;
    const int col0 = tall ? 0 : c0, col1 = tall ? m : min(c0 + S::kCols, n);
    const int units = max(0, (col1 - col0 + 7) / 8);
    const int count = max(0, row1 - row0) * units;
    for (int i0 = threadIdx.x; i0 < count; i0 += kUnits * kSmallThreads) {
      float u[kUnits][8] = {}, mom[kUnits][8];
#pragma unroll
      for (int q = 0; q < kUnits; ++q) {
        const int i = i0 + q * kSmallThreads;
        if (i >= count) break;
        const int r = row0 + i / units, c = col0 + i % units * 8;
        const int k8 = min(8, col1 - c);
        if (p.f32)
          load_grad<true>(p, z, r, c, k8, u[q]);
        else
          load_grad<false>(p, z, r, c, k8, u[q]);
        if (p.mom != nullptr)
          load_floats(p.mom + z * p.plane_m + r * p.ld_m + c, k8, p.vec, mom[q]);
      }
#pragma unroll
      for (int q = 0; q < kUnits; ++q) {
        const int i = i0 + q * kSmallThreads;
        if (i >= count) break;
        const int r = row0 + i / units, c = col0 + i % units * 8;
        if (p.mom != nullptr) {
          step_momentum(p, z, r, c, min(8, col1 - c), u[q], mom[q]);
          direction(p, u[q], mom[q]);
        }
        // whole units: past the matrix their elements are zeros
        float4* to = reinterpret_cast<float4*>(U + (tall ? (r - c0) * S::kPitchT + c
                                                         : r * S::kPitchU + c - c0));
        to[0] = make_float4(u[q][0], u[q][1], u[q][2], u[q][3]);
        to[1] = make_float4(u[q][4], u[q][5], u[q][6], u[q][7]);
      }
      float all;
      if (middle_squares(u, all)) {
        middle += all;
      } else {
        sum += squares_of(u);
        odd = true;
      }
    }
  }
  // (fp64 is slow: no more warps than it needs)
  if (__syncthreads_or(odd)) {
    s_part[threadIdx.x] = sum + middle;
    __syncthreads();
    sum = 0.0;
    if (warp == 0)
      for (int w = 0; w < kSmallWarps; ++w) sum += s_part[32 * w + lane];
  } else {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) middle += __shfl_xor_sync(0xFFFFFFFFu, middle, o);
    if (lane == 0) s_warp[warp] = middle;
    __syncthreads();
    if (warp == 0) sum = lane < kSmallWarps ? s_warp[lane] : 0.0f;
  }
  if (warp == 0) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
  }
  cluster_wait();                            // before anything goes to another CTA
  if (threadIdx.x < ctas) st_cluster_f64(mapa_shared(smem_u32(&s_norm[rank]), threadIdx.x), sum);
  cluster_sync();
  if (warp == 0) {
    sum = lane < static_cast<int>(ctas) ? s_norm[lane] : 0.0;
#pragma unroll
    for (int o = kMaxCluster / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    if (lane == 0) {
      const float f = static_cast<float>(sum);
      s_mul = f > 1e-28f && f < 1e36f
                  ? make_float2(p.x_scale / (sqrtf(f) + p.eps), 1.0f)
                  : norm_factors(sum, p.x_scale, p.eps);
    }
  }
  __syncthreads();
  const float2 mul = s_mul;

  // ---- X in the accumulators: 32 rows, 8 NB columns a warp
  const int xr0 = warp / S::kColWarps * 32, xc0 = warp % S::kColWarps * (8 * NB);
  const int gr = lane / 4, gc = lane % 4 * 2;
  float x[2][NB][4];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = xr0 + 16 * i + gr + 8 * h, c = xc0 + 8 * j + gc;
        float2 v;
        if (tall)
          v = make_float2(U[c * S::kPitchT + r], U[(c + 1) * S::kPitchT + r]);
        else
          v = *reinterpret_cast<const float2*>(U + r * S::kPitchU + c);
        x[i][j][2 * h] = v.x * mul.x * mul.y;
        x[i][j][2 * h + 1] = v.y * mul.x * mul.y;
      }
  cluster_arrive();                          // U may be written over, by other CTAs too
  __syncthreads();

  const float to_a = kOrthoScaleA / (p.x_scale * p.x_scale);
  const uint32_t x_at = smem_u32(X), a_at = smem_u32(A), b_at = smem_u32(B);
  // a warp's block of A and B
  const int ar0 = warp / 4 * (16 * MB), ac0 = warp % 4 * (16 * NB2);
  const int share = (MP + ctas - 1) / ctas;     // rows of A that a CTA adds up
  const int first = static_cast<int>(rank) * share;
  const int rows = max(0, min(share, MP - first));
  const uint32_t p_at = smem_u32(P), p_bar_at = smem_u32(&p_bar), a_bar_at = smem_u32(&a_bar);
  const float* received = reinterpret_cast<const float*>(smem + S::kRAt);
  for (int step = 0; step < g.steps; ++step) {
    // the operand
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < NB; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          *reinterpret_cast<uint32_t*>(X + (xr0 + 16 * i + gr + 8 * h) * S::kPitchX + xc0 + 8 * j +
                                       gc) = pack_half2(x[i][j][2 * h], x[i][j][2 * h + 1]);
    __syncthreads();
    float acc[MB][2 * NB2][4];
    rows_product<MB, NB2>(acc, x_at, S::kPitchX, ar0, ac0, S::kCols, lane);
    if (step == 0) cluster_wait();
    if (threadIdx.x == 0 && !s_abort) {
      if constexpr (S::kSend) mbar_arrive_expect_tx(&p_bar, ctas * rows * S::kPitchP * 4);
      mbar_arrive_expect_tx(&a_bar, MP * MP * 2);
    }
    // (everyone has read the last P and A: each CTA's part of A came after that, and
    // all of it was here)
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
      for (int j = 0; j < 2 * NB2; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          *reinterpret_cast<float2*>(P + (ar0 + 16 * i + gr + 8 * h) * S::kPitchP + ac0 + 8 * j +
                                     gc) = make_float2(acc[i][j][2 * h], acc[i][j][2 * h + 1]);
    if constexpr (S::kSend) {
      // rows to the CTA that adds them up
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncthreads();
      const int r = threadIdx.x * share;
      if (threadIdx.x < ctas && r < MP) {
        send(mapa_shared(smem_u32(received + rank * share * S::kPitchP), threadIdx.x),
             p_at + r * S::kPitchP * 4, min(share, MP - r) * S::kPitchP * 4,
             mapa_shared(p_bar_at, threadIdx.x));
      }
      wait_sent(&p_bar, step & 1, g.status, &s_abort);
    } else {
      cluster_sync();
    }
    // this CTA's rows of A, into everyone's
    for (int i = threadIdx.x; i < rows * (MP / 4); i += kSmallThreads) {
      const int r = i / (MP / 4), c = i % (MP / 4) * 4;
      float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (uint32_t q0 = 0; q0 < kMaxCluster; q0 += 4) {
        float4 w[4];
#pragma unroll
        for (uint32_t q = 0; q < 4; ++q) {
          if (q0 + q >= ctas) break;
          if constexpr (S::kSend)
            w[q] = *reinterpret_cast<const float4*>(received +
                                                    ((q0 + q) * share + r) * S::kPitchP + c);
          else
            w[q] = ld_cluster4(mapa_shared(p_at + ((first + r) * S::kPitchP + c) * 4, q0 + q));
        }
#pragma unroll
        for (uint32_t q = 0; q < 4; ++q) {
          if (q0 + q >= ctas) break;
          v.x += w[q].x;
          v.y += w[q].y;
          v.z += w[q].z;
          v.w += w[q].w;
        }
      }
      const uint32_t lo = pack_half2(v.x * to_a, v.y * to_a), hi = pack_half2(v.z * to_a, v.w * to_a);
      const uint32_t to = a_at + ((first + r) * S::kPitchA + c) * 2;
      for (uint32_t q = 0; q < ctas; ++q)
        st_async2(mapa_shared(to, q), lo, hi, mapa_shared(a_bar_at, q));
    }
    wait_sent(&a_bar, step & 1, g.status, &s_abort);
    // B
    rows_product<MB, NB2>(acc, a_at, S::kPitchA, ar0, ac0, MP, lane);
    const bool shifted = step + 2 >= g.steps;
    const float ca = g.b / kOrthoScaleA, caa = g.c / (kOrthoScaleA * kOrthoScaleA);
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
      for (int j = 0; j < 2 * NB2; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int r = ar0 + 16 * i + gr + 8 * h, c = ac0 + 8 * j + gc;
          const float2 in =
              __half22float2(*reinterpret_cast<const __half2*>(A + r * S::kPitchA + c));
          const float v0 = fmaf(in.x, ca, acc[i][j][2 * h] * caa);
          const float v1 = fmaf(in.y, ca, acc[i][j][2 * h + 1] * caa);
          *reinterpret_cast<uint32_t*>(B + r * S::kPitchA + c) = pack_half2(v0, v1);
          if (shifted && r == c) s_diag[r] = v0;
          if (shifted && r == c + 1) s_diag[r] = v1;
        }
    __syncthreads();
    float s = 0.0f;
    if (shifted) {
#pragma unroll
      for (int i = 0; i < MP; i += 32) s += s_diag[i + lane];   // (zero past the m-th)
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
      s /= static_cast<float>(m);
      if (threadIdx.x < m)
        B[threadIdx.x * S::kPitchA + threadIdx.x] = __float2half_rn(s_diag[threadIdx.x] - s);
      __syncthreads();
    }
    // X
    const float keep = g.a + s;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < NB; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) x[i][j][q] *= keep;
    const uint32_t left = b_at + ((xr0 + lane % 16) * S::kPitchA + lane / 16 * 8) * 2;
    const uint32_t right = x_at + (lane % 16 * S::kPitchX + xc0 + lane / 16 * 8) * 2;
#pragma unroll 2
    for (int k0 = 0; k0 < MP; k0 += 16) {
      uint32_t a[2][4];
      ldsm4(left + k0 * 2, a[0]);
      ldsm4(left + (16 * S::kPitchA + k0) * 2, a[1]);
#pragma unroll
      for (int j = 0; j < NB; j += 2) {
        uint32_t b[4];
        ldsm4_t(right + (k0 * S::kPitchX + 8 * j) * 2, b);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          mma16(x[i][j], a[i], b[0], b[1]);
          if (j + 1 < NB) mma16(x[i][j + 1 < NB ? j + 1 : j], a[i], b[2], b[3]);
        }
      }
    }
    __syncthreads();
  }

  // ---- the result, by way of shared memory along the caller's rows
  const float to_out = g.scale / p.x_scale;
  cluster_arrive();                          // nothing is sent any more
  __nv_bfloat16* Y = reinterpret_cast<__nv_bfloat16*>(smem);
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = xr0 + 16 * i + gr + 8 * h, c = xc0 + 8 * j + gc;
        const uint32_t two = pack_bf16x2(x[i][j][2 * h] * to_out, x[i][j][2 * h + 1] * to_out);
        if (tall) {
          uint16_t* y = reinterpret_cast<uint16_t*>(Y) + c * S::kPitchY + r;
          y[0] = static_cast<uint16_t>(two);
          y[S::kPitchY] = static_cast<uint16_t>(two >> 16);
        } else {
          *reinterpret_cast<uint32_t*>(Y + r * S::kPitchX + c) = two;
        }
      }
  __syncthreads();
  {
    const int row0 = tall ? c0 : 0, row1 = tall ? min(c0 + S::kCols, n) : m;
    const int col0 = tall ? 0 : c0, col1 = tall ? m : min(c0 + S::kCols, n);
    const int units = max(0, (col1 - col0 + 7) / 8);
    const int count = max(0, row1 - row0) * units;
    for (int i = threadIdx.x; i < count; i += kSmallThreads) {
      const int r = row0 + i / units, c = col0 + i % units * 8;
      __nv_bfloat16* dst = g.out + z * g.plane_out + r * g.ld_out + c;
      const uint4 v = *reinterpret_cast<const uint4*>(
          Y + (tall ? (r - c0) * S::kPitchY + c : r * S::kPitchX + c - c0));
      if (g.out_vec && c + 8 <= col1) {
        *reinterpret_cast<uint4*>(dst) = v;
      } else {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (c + k < col1)
            reinterpret_cast<uint16_t*>(dst)[k] = static_cast<uint16_t>(w[k / 2] >> 16 * (k % 2));
      }
    }
  }
  cluster_wait();
}

template <int MP, int NB>
cudaLaunchConfig_t config_of(int batch, int ctas, cudaStream_t s, cudaLaunchAttribute* attr) {
  attr->id = cudaLaunchAttributeClusterDimension;
  attr->val.clusterDim.x = ctas;
  attr->val.clusterDim.y = attr->val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(batch) * ctas);
  cfg.blockDim = dim3(kSmallThreads);
  cfg.dynamicSmemBytes = SmallShape<MP, NB>::kBytes;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cfg;
}

template <int MP, int NB>
cudaError_t prepare_shape() {
  cudaError_t err = cudaFuncSetAttribute(k_ortho_small<MP, NB>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         SmallShape<MP, NB>::kBytes);
  if (err == cudaSuccess)
    err = cudaFuncSetAttribute(k_ortho_small<MP, NB>, cudaFuncAttributeNonPortableClusterSizeAllowed,
                               1);
  return err;
}

// Whether this GPU holds `batch` clusters of that many CTAs at once.  (GPCs differ in
// their SMs from one GPU to the next, so it is asked, once a device.)
template <int MP, int NB>
bool holds(int batch, int ctas) {
  if (ctas <= kPortable) return true;
  constexpr int kDevices = 64;
  static std::atomic<int> known[kDevices][kMaxCluster - kPortable];   // clusters, and one
  int dev;
  if (cudaGetDevice(&dev) != cudaSuccess) return false;
  std::atomic<int>* have = dev < kDevices ? &known[dev][ctas - kPortable - 1] : nullptr;
  int clusters = have != nullptr ? have->load(std::memory_order_relaxed) - 1 : -1;
  if (clusters < 0) {
    cudaLaunchAttribute attr;
    const cudaLaunchConfig_t cfg = config_of<MP, NB>(batch, ctas, nullptr, &attr);
    if (prepare_shape<MP, NB>() != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&clusters, k_ortho_small<MP, NB>, &cfg) != cudaSuccess) {
      cudaGetLastError();        // the question's: fewer CTAs do
      clusters = 0;
    }
    if (have != nullptr) have->store(clusters + 1, std::memory_order_relaxed);
  }
  return clusters >= batch;
}

template <int MP, int NB>
cudaError_t launch_shape(const SmallOrthoArgs& g, int ctas, cudaStream_t s) {
  const cudaError_t err = prepare_shape<MP, NB>();
  if (err != cudaSuccess) return err;
  cudaLaunchAttribute attr;
  const cudaLaunchConfig_t cfg = config_of<MP, NB>(g.in.batch, ctas, s, &attr);
  return cudaLaunchKernelEx(&cfg, k_ortho_small<MP, NB>, g);
}

// The fewest columns a CTA (8 NB for each of its warps along the columns) that leave a
// matrix in one cluster and all clusters on the GPU at once: more CTAs have shorter
// products, fewer have less to exchange.  More than eight where they keep 64 columns
// (16 instead of 8: 64 x 2048 with a momentum 29.2 -> 24.6 us, 128 x 2048 72 -> 59,
// 128 x 1024 53 -> 52; with 32 columns each 128 x 512 46 -> 50).
template <int MP, int NB>
cudaError_t launch_rows(const SmallOrthoArgs& g, int n, int sms, cudaStream_t s) {
  const int ctas = (n + SmallShape<MP, NB>::kCols - 1) / SmallShape<MP, NB>::kCols;
  if constexpr (NB < 8) {
    const int most = SmallShape<MP, NB>::kCols >= 64 ? kMaxCluster : kPortable;
    if (ctas > 1 && (ctas > most || static_cast<long long>(ctas) * g.in.batch > sms ||
                     !holds<MP, NB>(g.in.batch, ctas)))
      return launch_rows<MP, 2 * NB>(g, n, sms, s);
  }
  return launch_shape<MP, NB>(g, ctas, s);
}

}  // namespace

bool small_ortho(int rows, int cols) {
  const int m = rows < cols ? rows : cols, n = rows < cols ? cols : rows;
  if (m <= 64) return n <= kPortable * SmallShape<64, 8>::kCols;
  return m <= 128 && n <= kPortable * SmallShape<128, 8>::kCols;
}

cudaError_t launch_small_ortho(const SmallOrthoArgs& g, int sms, cudaStream_t s) {
  const int m = g.in.rows < g.in.cols ? g.in.rows : g.in.cols;
  const int n = g.in.rows < g.in.cols ? g.in.cols : g.in.rows;
  return m <= 64 ? launch_rows<64, 1>(g, n, sms, s) : launch_rows<128, 1>(g, n, sms, s);
}

}  // namespace moe
