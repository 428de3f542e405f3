// Orthogonalised updates: what the general kernels (moe_ortho.cu) and those of
// small matrices (moe_ortho_small.cu) share.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "moe_f2.cuh"
#include "moe_internal.h"
#include "moe_ptx.cuh"

namespace moe {

constexpr float kOrthoScaleA = 4096.0f;        // A's entries are at most 4: A is held times this

// What the preparation of X reads and writes.
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
  float* state;
  long long ld_x, plane_x, plane_s;
  unsigned int* done;          // k_ortho_steps' counts, set to zero
};

// 8 floats of a row from c on, n of them where they are not aligned.
__device__ __forceinline__ void load_floats(const float* src, int n, bool vec, float (&v)[8]) {
  if (vec) {
    const float4* q = reinterpret_cast<const float4*>(src);
    const float4 x = q[0], y = q[1];
    v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
    v[4] = y.x, v[5] = y.y, v[6] = y.z, v[7] = y.w;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < n ? src[i] : 0.0f;
  }
}

template <bool F32>
__device__ __forceinline__ void load_grad(const PrepArgs& p, int z, int r, int c, int n,
                                          float (&g)[8]) {
  const long long at = z * p.plane_g + r * p.ld_g + c;
  if constexpr (F32) {
    load_floats(static_cast<const float*>(p.grad) + at, n, p.vec, g);
  } else {
    const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(p.grad) + at;
    if (p.vec) {
      const uint4 x = *reinterpret_cast<const uint4*>(src);
      const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        g[2 * i] = bf16_lo(w[i]);
        g[2 * i + 1] = bf16_hi(w[i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) g[i] = i < n ? __bfloat162float(src[i]) : 0.0f;
    }
  }
}

// The new momentum of 8 elements from the old one, in place and stored.
__device__ __forceinline__ void step_momentum(const PrepArgs& p, int z, int r, int c, int n,
                                              const float (&g)[8], float (&m)[8]) {
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

// U of the gradient g and the new momentum, into g.
__device__ __forceinline__ void direction(const PrepArgs& p, float (&g)[8], const float (&m)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) g[i] = p.nesterov ? fmaf(p.mu, m[i], p.nu * g[i]) : m[i];
}

// Squares of 8 N values in fp32; false where their sum is not in its middle range.
template <int N>
__device__ __forceinline__ bool middle_squares(const float (&u)[N][8], float& all) {
  float sq[N];
  all = 0.0f;
#pragma unroll
  for (int q = 0; q < N; ++q) {
    sq[q] = 0.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k) sq[q] = fmaf(u[q][k], u[q][k], sq[q]);
    all += sq[q];
  }
  if (all > 1e-30f && all < 1e30f) return true;
  bool zeros = all == 0.0f;          // a sum of 0 is one of zeros, or of squares below fp32's range
#pragma unroll
  for (int q = 0; q < N; ++q)
#pragma unroll
    for (int k = 0; k < 8; ++k) zeros = zeros && u[q][k] == 0.0f;
  return zeros;
}

// The same in fp64 where fp32 does not hold them.  (One fp64 addition for them all:
// this GPU's rate of those is 1/64.)
template <int N>
__device__ __forceinline__ double squares_of(const float (&u)[N][8]) {
  float all;
  if (middle_squares(u, all)) return all;
  double sum = 0.0;
#pragma unroll
  for (int q = 0; q < N; ++q)
#pragma unroll
    for (int k = 0; k < 8; ++k) sum += static_cast<double>(u[q][k]) * u[q][k];
  return sum;
}

// What U is multiplied by, x_scale / (|U| + eps), as two factors: with a norm and an
// eps near fp32's smallest the one number would be inf, and a zero matrix NaN.
__device__ __forceinline__ float2 norm_factors(double squares, float x_scale, float eps) {
  const double f = x_scale / (sqrt(squares) + eps);     // at most 2^14 / 2^-149
  return f > 1e38 ? make_float2(static_cast<float>(f * 0x1p-64), 0x1p64f)
                  : make_float2(static_cast<float>(f), 1.0f);
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Small matrices (moe_ortho_small.cu): whether the kernel that keeps a matrix in
// a cluster's registers takes this size, and its launch.
struct SmallOrthoArgs {
  PrepArgs in;
  __nv_bfloat16* out;
  long long ld_out, plane_out;
  int out_vec;                 // out's rows may be written 8 elements at a time
  int steps;
  float a, b, c, scale;
  int* status;
};
bool small_ortho(int rows, int cols);
cudaError_t launch_small_ortho(const SmallOrthoArgs& args, int sms, cudaStream_t s);

}  // namespace moe
