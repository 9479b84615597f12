// Residual addition and root-mean-square norm, with an optional block-FP8 copy of the result.
//
//   h[t]  = RN(x[t] + residual[t])                    (the stored residual stream; h = x without a residual)
//   n[t]  = h[t] * rsqrt(mean_j h[t, j]^2 + eps) * gamma
//   y[t]  = RN(n[t]),   s[t, g] = RN(amax_g |n| / 448),   code = E4M3_satfinite(RN(n / s)), 0 where s == 0
// for the 1 x 128 groups g of a row: the activation format of the block-FP8 shared expert (segemm.cu). The
// codes are taken from n in fp32, before the rounding to y's type, so they carry one rounding, not two.
//
// The sum of squares and the statistics are fp32; h is rounded to its storage type first, so the norm is
// that of the stream a later layer reads back.
//
// Bound by memory: a row is read and written once. One CTA takes a row.
#include "common.cuh"
#include "dense.cuh"
#include "internal.h"

namespace fp4moe {
namespace {

constexpr int NORM_THREADS = 256;

// Sum over the CTA, the same value in every thread.
__device__ __forceinline__ float cta_sum(float v, float* s_red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  if ((threadIdx.x & 31) == 0) s_red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.0f;
  for (int i = 0; i < (int)blockDim.x / 32; ++i) v += s_red[i];
  return v;
}

// Any width, any alignment: element accesses, and the row is read again for its second use. A warp takes
// whole 128-element groups, four elements a lane (lane, lane + 32, ...).
template <typename T>
__global__ void __launch_bounds__(NORM_THREADS)
    add_rmsnorm_any_kernel(int H, const T* x, const T* residual, const T* __restrict__ gamma, float eps, T* h_out,
                           T* y, uint8_t* codes, float* scales, int64_t scale_stride) {
  __shared__ float s_red[NORM_THREADS / 32];
  pdl_wait();
  pdl_trigger();
  const size_t row = (size_t)blockIdx.x * H;
  float ss = 0.0f;
  for (int j = threadIdx.x; j < H; j += NORM_THREADS) {
    float h = to_f32(x[row + j]);
    if (residual != nullptr) h = to_f32(from_f32<T>(__fadd_rn(h, to_f32(residual[row + j]))));
    ss = fmaf(h, h, ss);
  }
  ss = cta_sum(ss, s_red);
  const float rstd = __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(__fdiv_rn(ss, (float)H), eps)));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int g = warp; g * 128 < H; g += NORM_THREADS / 32) {
    float n[4], a = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int j = g * 128 + 32 * i + lane;
      n[i] = 0.0f;
      if (j < H) {
        float h = to_f32(x[row + j]);
        if (residual != nullptr) {
          const T r = from_f32<T>(__fadd_rn(h, to_f32(residual[row + j])));
          h = to_f32(r);
          h_out[row + j] = r;
        }
        n[i] = h * rstd * (gamma != nullptr ? to_f32(gamma[j]) : 1.0f);
        if (y != nullptr) y[row + j] = from_f32<T>(n[i]);
      }
      a = fmax_nan(a, fabsf(n[i]));  // a NaN takes its whole group along: NaN scale, NaN codes
    }
    if (codes != nullptr) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) a = fmax_nan(a, __shfl_xor_sync(0xFFFFFFFFu, a, o));
      const float s = __fdiv_rn(a, 448.0f);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int j = g * 128 + 32 * i + lane;
        if (j < H) codes[row + j] = s == 0.0f ? 0 : (uint8_t)cvt_e4m3x2(__fdiv_rn(n[i], s), 0.0f);
      }
      if (lane == 0) scales[(size_t)g * scale_stride + blockIdx.x] = s;
    }
  }
}

template <typename T>
fp4moe_status norm_launch(int32_t rows, int32_t H, const void* x, const void* residual, const void* gamma, float eps,
                          void* h_out, void* y, uint8_t* codes, float* scales, int64_t scale_stride,
                          cudaStream_t st) {
  const cudaError_t r =
      launch_pdl(add_rmsnorm_any_kernel<T>, dim3((unsigned)rows), dim3(NORM_THREADS), 0, st, H,
                 static_cast<const T*>(x), static_cast<const T*>(residual), static_cast<const T*>(gamma), eps,
                 static_cast<T*>(h_out), static_cast<T*>(y), codes, scales, scale_stride);
  return r == cudaSuccess ? FP4MOE_OK : FP4MOE_CUDA_ERROR;
}

}  // namespace

fp4moe_status add_rmsnorm_launch(int32_t dtype, int32_t rows, int32_t H, const void* x, const void* residual,
                                 const void* gamma, float eps, void* h_out, void* y, uint8_t* codes, float* scales,
                                 int64_t scale_stride, cudaStream_t st) {
  switch (dtype) {
    case FP4MOE_BF16:
      return norm_launch<__nv_bfloat16>(rows, H, x, residual, gamma, eps, h_out, y, codes, scales, scale_stride, st);
    case FP4MOE_FP16:
      return norm_launch<__half>(rows, H, x, residual, gamma, eps, h_out, y, codes, scales, scale_stride, st);
    default:
      return norm_launch<float>(rows, H, x, residual, gamma, eps, h_out, y, codes, scales, scale_stride, st);
  }
}

}  // namespace fp4moe
