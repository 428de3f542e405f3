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
  unsigned int* done;          // [batch][3], set to zero
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

// Squares of 8 values: in fp32, and in fp64 where their sum leaves fp32's middle
// range.
__device__ __forceinline__ double squares_of(const float (&u)[8]) {
  float sq = 0.0f;
#pragma unroll
  for (int k = 0; k < 8; ++k) sq = fmaf(u[k], u[k], sq);
  if (sq > 1e-30f && sq < 1e30f) return sq;
  double sum = 0.0;
#pragma unroll
  for (int k = 0; k < 8; ++k) sum += static_cast<double>(u[k]) * u[k];
  return sum;
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
};
bool small_ortho(int rows, int cols);
cudaError_t launch_small_ortho(const SmallOrthoArgs& args, int sms, cudaStream_t s);

}  // namespace moe
