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
// so two cluster barriers a step, no access to global memory between the read of
// the gradient and the write of the result, and no state but registers.  Operands
// and rounding are those of moe_ortho.cu.  These sizes are bound by latency, of
// barriers and of chains of small products, which mma.sync starts and ends in tens
// of cycles; a tcgen05 tile would be mostly empty at m = 64 and has to come back
// from TMEM each time (64 x 2048: 15 products of the general kernel took 139 us).
#include <math.h>

#include "moe_ortho.cuh"

namespace moe {
namespace {

constexpr int kSmallThreads = 512;
constexpr int kSmallWarps = 16;
constexpr int kMaxCluster = 8;                 // what every GPC holds

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

__device__ __forceinline__ void st_cluster2(uint32_t addr, uint32_t lo, uint32_t hi) {
  asm volatile("st.shared::cluster.v2.b32 [%0], {%1, %2};" ::"r"(addr), "r"(lo), "r"(hi)
               : "memory");
}

__device__ __forceinline__ void st_cluster_f64(uint32_t addr, double v) {
  asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(addr), "d"(v) : "memory");
}

// The two halves of cluster_sync(): here only to know that every CTA has started.
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
  static constexpr int kPitchU = kCols + 1;              // floats, of the gradient's stage
  static constexpr int kX = MP * kPitchX * 2;
  static constexpr int kA = MP * kPitchA * 2;
  static constexpr int kP = MP * kPitchP * 4;
  static constexpr int kU = MP * kPitchU * 4;
  static constexpr int kBytes = (kX + 2 * kA + kP > kU ? kX + 2 * kA + kP : kU);
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
#pragma unroll 2
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
  __shared__ double s_norm[kMaxCluster];
  __shared__ double s_warp[kSmallWarps];
  __shared__ float s_diag[MP];
  __half* X = reinterpret_cast<__half*>(smem);
  __half* A = reinterpret_cast<__half*>(smem + S::kX);
  __half* B = reinterpret_cast<__half*>(smem + S::kX + S::kA);
  float* P = reinterpret_cast<float*>(smem + S::kX + 2 * S::kA);
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

  cluster_arrive();
  // ---- the gradient and the momentum: this CTA's columns of U, and their squares
  double sum = 0.0;
  {
    for (int i = threadIdx.x; i < S::kU / 4; i += kSmallThreads) U[i] = 0.0f;
    __syncthreads();
    // along the caller's rows, 8 at a time: rows of this CTA's part
    const int row0 = tall ? c0 : 0, row1 = tall ? min(c0 + S::kCols, n) : m;
    const int col0 = tall ? 0 : c0, col1 = tall ? m : min(c0 + S::kCols, n);
    const int units = max(0, (col1 - col0 + 7) / 8);
    const int count = max(0, row1 - row0) * units;
    for (int i = threadIdx.x; i < count; i += kSmallThreads) {
      const int r = row0 + i / units, c = col0 + i % units * 8;
      const int k8 = min(8, col1 - c);
      float u1[1][8];
      float (&u)[8] = u1[0];
      if (p.f32)
        load_grad<true>(p, z, r, c, k8, u);
      else
        load_grad<false>(p, z, r, c, k8, u);
      if (p.mom != nullptr) {
        float mom[8];
        load_floats(p.mom + z * p.plane_m + r * p.ld_m + c, k8, p.vec, mom);
        step_momentum(p, z, r, c, k8, u, mom);
        direction(p, u, mom);
      }
      sum += squares_of(u1);
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (c + k < col1) {
          const int xr = tall ? c + k : r, xc = tall ? r - c0 : c + k - c0;
          U[xr * S::kPitchU + xc] = u[k];
        }
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
  if (lane == 0) s_warp[warp] = sum;
  __syncthreads();
  cluster_wait();                            // before anything goes to another CTA
  if (threadIdx.x < ctas) {
    sum = 0.0;
    for (int w = 0; w < kSmallWarps; ++w) sum += s_warp[w];
    st_cluster_f64(mapa_shared(smem_u32(&s_norm[rank]), threadIdx.x), sum);
  }
  cluster_sync();
  sum = 0.0;
  for (uint32_t r = 0; r < ctas; ++r) sum += s_norm[r];
  const float mul = static_cast<float>(p.x_scale / (sqrt(sum) + p.eps));

  // ---- X in the accumulators: 32 rows, 8 NB columns a warp
  const int xr0 = warp / S::kColWarps * 32, xc0 = warp % S::kColWarps * (8 * NB);
  const int gr = lane / 4, gc = lane % 4 * 2;
  float x[2][NB][4];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        x[i][j][q] = U[(xr0 + 16 * i + gr + q / 2 * 8) * S::kPitchU + xc0 + 8 * j + gc + q % 2] * mul;
  __syncthreads();

  const float to_a = kOrthoScaleA / (p.x_scale * p.x_scale);
  const uint32_t x_at = smem_u32(X), a_at = smem_u32(A), b_at = smem_u32(B);
  // a warp's block of A and B
  const int ar0 = warp / 4 * (16 * MB), ac0 = warp % 4 * (16 * NB2);
  const int share = (MP + ctas - 1) / ctas;     // rows of A that a CTA adds up
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
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
      for (int j = 0; j < 2 * NB2; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          *reinterpret_cast<float2*>(P + (ar0 + 16 * i + gr + 8 * h) * S::kPitchP + ac0 + 8 * j +
                                     gc) = make_float2(acc[i][j][2 * h], acc[i][j][2 * h + 1]);
    cluster_sync();
    // this CTA's rows of A, into everyone's
    const int first = static_cast<int>(rank) * share;
    const int rows = min(share, MP - first);
    for (int i = threadIdx.x; i < rows * (MP / 4); i += kSmallThreads) {
      const int r = first + i / (MP / 4), c = i % (MP / 4) * 4;
      const uint32_t at = smem_u32(P + r * S::kPitchP + c);
      float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      for (uint32_t q = 0; q < ctas; ++q) {
        const float4 w = ld_cluster4(mapa_shared(at, q));
        v.x += w.x;
        v.y += w.y;
        v.z += w.z;
        v.w += w.w;
      }
      const uint32_t lo = pack_half2(v.x * to_a, v.y * to_a), hi = pack_half2(v.z * to_a, v.w * to_a);
      const uint32_t to = a_at + (r * S::kPitchA + c) * 2;
      for (uint32_t q = 0; q < ctas; ++q) st_cluster2(mapa_shared(to, q), lo, hi);
    }
    cluster_sync();
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
  __nv_bfloat16* Y = reinterpret_cast<__nv_bfloat16*>(smem);
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        *reinterpret_cast<uint32_t*>(Y + (xr0 + 16 * i + gr + 8 * h) * S::kPitchX + xc0 + 8 * j +
                                     gc) =
            pack_bf16x2(x[i][j][2 * h] * to_out, x[i][j][2 * h + 1] * to_out);
  __syncthreads();
  {
    const int row0 = tall ? c0 : 0, row1 = tall ? min(c0 + S::kCols, n) : m;
    const int col0 = tall ? 0 : c0, col1 = tall ? m : min(c0 + S::kCols, n);
    const int units = max(0, (col1 - col0 + 7) / 8);
    const int count = max(0, row1 - row0) * units;
    for (int i = threadIdx.x; i < count; i += kSmallThreads) {
      const int r = row0 + i / units, c = col0 + i % units * 8;
      __nv_bfloat16* dst = g.out + z * g.plane_out + r * g.ld_out + c;
      uint16_t v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int xr = tall ? c + k : r, xc = tall ? r - c0 : c + k - c0;
        // (a unit may reach past the short side, within the padded rows)
        v[k] = reinterpret_cast<const uint16_t*>(Y)[xr * S::kPitchX + xc];
      }
      if (g.out_vec && c + 8 <= col1) {
        *reinterpret_cast<uint4*>(dst) =
            make_uint4(v[0] | static_cast<uint32_t>(v[1]) << 16, v[2] | static_cast<uint32_t>(v[3]) << 16,
                       v[4] | static_cast<uint32_t>(v[5]) << 16, v[6] | static_cast<uint32_t>(v[7]) << 16);
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (c + k < col1) reinterpret_cast<uint16_t*>(dst)[k] = v[k];
      }
    }
  }
}

template <int MP, int NB>
cudaError_t launch_shape(const SmallOrthoArgs& g, int ctas, cudaStream_t s) {
  using S = SmallShape<MP, NB>;
  cudaError_t err = cudaFuncSetAttribute(
      k_ortho_small<MP, NB>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kBytes);
  if (err != cudaSuccess) return err;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = ctas;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(g.in.batch) * ctas);
  cfg.blockDim = dim3(kSmallThreads);
  cfg.dynamicSmemBytes = S::kBytes;
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_ortho_small<MP, NB>, g);
}

// The fewest columns a CTA that leave a matrix in kMaxCluster CTAs, and all
// matrices' CTAs on the GPU at once where that is to be had: more CTAs have
// shorter products, fewer have less to exchange.
template <int MP>
cudaError_t launch_rows(const SmallOrthoArgs& g, int n, int sms, cudaStream_t s) {
  constexpr int unit = SmallShape<MP, 1>::kCols;
  int nb = 1;
  while (nb < 8) {
    const int ctas = (n + nb * unit - 1) / (nb * unit);
    if (ctas <= kMaxCluster && static_cast<long long>(ctas) * g.in.batch <= sms) break;
    if (ctas == 1) break;
    nb *= 2;
  }
  const int ctas = (n + nb * unit - 1) / (nb * unit);
  switch (nb) {
    case 1: return launch_shape<MP, 1>(g, ctas, s);
    case 2: return launch_shape<MP, 2>(g, ctas, s);
    case 4: return launch_shape<MP, 4>(g, ctas, s);
    default: return launch_shape<MP, 8>(g, ctas, s);
  }
}

}  // namespace

bool small_ortho(int rows, int cols) {
  const int m = rows < cols ? rows : cols, n = rows < cols ? cols : rows;
  if (m <= 64) return n <= kMaxCluster * SmallShape<64, 8>::kCols;
  return m <= 128 && n <= kMaxCluster * SmallShape<128, 8>::kCols;
}

cudaError_t launch_small_ortho(const SmallOrthoArgs& g, int sms, cudaStream_t s) {
  const int m = g.in.rows < g.in.cols ? g.in.rows : g.in.cols;
  const int n = g.in.rows < g.in.cols ? g.in.cols : g.in.rows;
  return m <= 64 ? launch_rows<64>(g, n, sms, s) : launch_rows<128>(g, n, sms, s);
}

}  // namespace moe
