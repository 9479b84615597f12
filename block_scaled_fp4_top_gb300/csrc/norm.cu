// Residual addition and root-mean-square norm, with an optional block-FP8 copy of the result.
//
//   h[t]  = RN(x[t] + residual[t])                    (the stored residual stream; h = x without a residual)
//   n[t]  = h[t] * rsqrt(mean_j h[t, j]^2 + eps) * gamma
//   y[t]  = RN(n[t]),   s[t, g] = RN(amax_g |n| / 448),   code = E4M3_satfinite(n / s), 0 where s == 0
// for the 1 x 128 groups g of a row: the activation format of the block-FP8 shared expert (segemm.cu). The
// codes are taken from n in fp32, before the rounding to y's type, so they carry one rounding, not two.
//
// The sum of squares and the statistics are fp32; h is rounded to its storage type first, so the norm is
// that of the stream a later layer reads back.
//
// Bound by memory: a row is read and written once. One CTA takes a row and, where it fits, keeps
// it in registers between the two uses: NV 16-byte vectors a thread. Few rows leave the device empty and the time is one trip to memory, a reduction and a trip back, so
// they take the most threads (NV = 1); many rows take two vectors a thread.
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

// n / s as (n * up) * inv, to within two units of fp32's last place; 0 where s == 0. One reciprocal serves a group:
// exact enough for a value that E4M3 rounds to four bits. Below 2^-120 it would overflow, so n and s are first
// scaled up by 2^100, exactly (a subnormal n included).
struct Fp8Scale {
  float up, inv;
};
__device__ __forceinline__ Fp8Scale fp8_scale(float s) {
  if (s < 0x1p-120f) return s == 0.0f ? Fp8Scale{0.0f, 0.0f} : Fp8Scale{0x1p100f, __frcp_rn(s * 0x1p100f)};
  return Fp8Scale{1.0f, __frcp_rn(s)};
}
// N codes of the quotients q.
template <int N>
__device__ __forceinline__ void make_codes(uint32_t (&w)[N / 4], const float (&q)[N]) {
#pragma unroll
  for (int k = 0; k < N; k += 4) w[k / 4] = cvt_e4m3x2(q[k], q[k + 1]) | (cvt_e4m3x2(q[k + 2], q[k + 3]) << 16);
}
// N codes at p (aligned to N bytes).
template <int N>
__device__ __forceinline__ void store_codes(uint8_t* p, const uint32_t (&w)[N / 4]) {
  if constexpr (N == 8)
    *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
  else
    *reinterpret_cast<uint32_t*>(p) = w[0];
}

// Widths too large for a CTA's registers: element accesses, and the row is read again for its second use. A warp takes whole 128-element
// groups, four elements a lane (lane, lane + 32, ...).
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
      const Fp8Scale f = fp8_scale(s);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int j = g * 128 + 32 * i + lane;
        if (j < H) codes[row + j] = (uint8_t)cvt_e4m3x2(n[i] * f.up * f.inv, 0.0f);
      }
      if (lane == 0) scales[(size_t)g * scale_stride + blockIdx.x] = s;
    }
  }
}

// 16 bytes of a row. Plain loads, not the read-only path: an output may be the same buffer. Each element is read
// and written by one thread, in that order.
__device__ __forceinline__ uint4 ld_vec(const void* p) {
  uint4 q;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(q.x), "=r"(q.y), "=r"(q.z), "=r"(q.w)
               : "l"(p));
  return q;
}

// 16 bytes from byte 16 - back of the 32 bytes (prev, cur); back is the same in the whole CTA, 0 .. 14 and even.
__device__ __forceinline__ uint4 shifted(uint4 prev, uint4 cur, int back) {
  if (back == 0) return cur;
  uint32_t w[8] = {prev.x, prev.y, prev.z, prev.w, cur.x, cur.y, cur.z, cur.w};
  shift_words<8, 4>(w, 16 - back);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Vector q of a row, in a thread's slot i, is q = i * blockDim + threadIdx.
//
// SHIFT: rows whose length no vector divides start at any element of a vector. x, residual, h_out and y then
// all start at the same one (their bases are 16-byte aligned), and so do the codes in units of N bytes. So the
// kernel cuts a row at the addresses that N divides: vector q holds elements N q - off .. N q - off + N - 1,
// off = the row's first element modulo N, and only the first and the last vector of a row are partly outside.
// gamma starts aligned, so its N elements come from two vectors, shifted into place. The vectors of one FP8
// group are 128 / N neighbouring lanes, except that the first `off` elements of the first of them belong to
// the group before: their maximum goes through shared memory (s_head), like the group's own (s_main).
// Elements outside the row are zeros all the way (a NaN statistic makes them NaN, and then its row is, too).
template <typename T, int NV, bool SHIFT>
__global__ void __launch_bounds__(1024)
    add_rmsnorm_vec_kernel(int H, const T* x, const T* residual, const T* __restrict__ gamma, float eps, T* h_out,
                           T* y, uint8_t* codes, float* scales, int64_t scale_stride) {
  constexpr int N = 16 / (int)sizeof(T), LANES = 128 / N;
  __shared__ float s_red[32];
  __shared__ float s_main[SHIFT ? NV * 1024 / LANES : 1], s_head[SHIFT ? NV * 1024 / LANES + 1 : 1];
  __shared__ Fp8Scale s_scale[SHIFT ? NV * 1024 / LANES : 1];
  pdl_wait();
  pdl_trigger();
  const size_t row = (size_t)blockIdx.x * H;
  const int off = SHIFT ? (int)(row % N) : 0;
  // first element of slot i's vector; whole: every element is in the row; edge: some are
  auto at = [&](int i) { return (i * (int)blockDim.x + (int)threadIdx.x) * N - off; };
  auto whole = [&](int j) { return SHIFT ? (j >= 0 && j + N <= H) : j < H; };
  auto edge = [&](int j) { return SHIFT && j < H && (j < 0 || j + N > H); };
  auto inside = [&](int j, int k) { return (unsigned)(j + k) < (unsigned)H; };
  auto store = [&](T* p, int j, uint4 v) {
    if (whole(j)) {
      *reinterpret_cast<uint4*>(p + row + j) = v;
    } else if (edge(j)) {
      alignas(16) T e[N];
      *reinterpret_cast<uint4*>(e) = v;
#pragma unroll
      for (int k = 0; k < N; ++k)
        if (inside(j, k)) p[row + j + k] = e[k];
    }
  };
  // Every load of the row is issued before the first is waited for. gamma waits until x and the residual are
  // joined where its registers would cost occupancy: 8192 x 4096 bf16 without a residual 24.7 against 29.7 us.
  constexpr bool kGammaFirst = SHIFT || NV == 1;
  uint4 hv[NV], rv[NV], gv[NV], gp[SHIFT ? NV : 1];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int j = at(i);
    hv[i] = rv[i] = gv[i] = make_uint4(0, 0, 0, 0);
    if (whole(j)) hv[i] = ld_vec(x + row + j);
    if (residual != nullptr && whole(j)) rv[i] = ld_vec(residual + row + j);
    if (kGammaFirst && gamma != nullptr && j + off + N <= H) gv[i] = __ldg(reinterpret_cast<const uint4*>(gamma + j + off));
    if constexpr (SHIFT) {
      gp[i] = make_uint4(0, 0, 0, 0);
      if (gamma != nullptr && off > 0 && j + off > 0 && j + off + N <= H)
        gp[i] = __ldg(reinterpret_cast<const uint4*>(gamma + j + off - N));
    }
  }
  if constexpr (SHIFT) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int j = at(i);
      gv[i] = shifted(gp[i], gv[i], off * (int)sizeof(T));
      if (j < H && (j < 0 || j + off + N > H)) {  // the row's first or last elements, or gamma's last
        alignas(16) T ex[N], er[N], eg[N];
#pragma unroll
        for (int k = 0; k < N; ++k) {
          const bool in = inside(j, k);
          ex[k] = in ? x[row + j + k] : from_f32<T>(0.0f);
          er[k] = in && residual != nullptr ? residual[row + j + k] : from_f32<T>(0.0f);
          eg[k] = in && gamma != nullptr ? gamma[j + k] : from_f32<T>(0.0f);
        }
        hv[i] = *reinterpret_cast<const uint4*>(ex);
        rv[i] = *reinterpret_cast<const uint4*>(er);
        gv[i] = *reinterpret_cast<const uint4*>(eg);
      }
    }
  }
  if (residual != nullptr) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float h[N], r[N];
      unpack<T>(hv[i], h);
      unpack<T>(rv[i], r);
#pragma unroll
      for (int k = 0; k < N; ++k) h[k] = __fadd_rn(h[k], r[k]);
      hv[i] = pack<T>(h);
      store(h_out, at(i), hv[i]);
    }
  }
  if constexpr (!kGammaFirst) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (gamma != nullptr && at(i) < H) gv[i] = __ldg(reinterpret_cast<const uint4*>(gamma + at(i)));
  }
  float ss = 0.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    float h[N];
    unpack<T>(hv[i], h);
#pragma unroll
    for (int k = 0; k < N; ++k) ss = fmaf(h[k], h[k], ss);
  }
  ss = cta_sum(ss, s_red);
  const float rstd = __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(__fdiv_rn(ss, (float)H), eps)));

  // fmax_nan: a NaN takes its whole group along (NaN scale, NaN codes)
  float n[NV][N];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int j = at(i);
    float a = 0.0f, head = 0.0f;
    unpack<T>(hv[i], n[i]);
#pragma unroll
    for (int k = 0; k < N; ++k) n[i][k] *= rstd;
    if (gamma != nullptr) {
      float g[N];
      unpack<T>(gv[i], g);
#pragma unroll
      for (int k = 0; k < N; ++k) n[i][k] *= g[k];
    }
    if (y != nullptr) store(y, j, pack<T>(n[i]));
    if (codes != nullptr) {
#pragma unroll
      for (int k = 0; k < N; ++k) {
        if (SHIFT && k < off)
          head = fmax_nan(head, fabsf(n[i][k]));
        else
          a = fmax_nan(a, fabsf(n[i][k]));
      }
      const bool first = (j + off) % 128 == 0;
      if (SHIFT && !first) a = fmax_nan(a, head);
#pragma unroll
      for (int o = LANES / 2; o > 0; o >>= 1) a = fmax_nan(a, __shfl_xor_sync(0xFFFFFFFFu, a, o));
      if constexpr (SHIFT) {
        if (first) {
          s_main[(j + off) / 128] = a;
          s_head[(j + off) / 128] = head;
        }
      } else if (j < H) {
        const float s = __fdiv_rn(a, 448.0f);
        const Fp8Scale f = fp8_scale(s);
        uint32_t w[N / 4];
#pragma unroll
        for (int k = 0; k < N; ++k) n[i][k] = n[i][k] * f.up * f.inv;
        make_codes<N>(w, n[i]);
        store_codes<N>(codes + row + j, w);
        if (first) scales[(size_t)(j / 128) * scale_stride + blockIdx.x] = s;
      }
    }
  }
  if constexpr (SHIFT) {
    if (codes == nullptr) return;
    const int G = (H + 127) / 128;
    if (threadIdx.x == 0) s_head[NV * (int)blockDim.x / LANES] = 0.0f;  // no vector follows the last group
    __syncthreads();
    for (int g = threadIdx.x; g < G; g += blockDim.x) {  // one thread a group
      const float s = __fdiv_rn(fmax_nan(s_main[g], s_head[g + 1]), 448.0f);
      scales[(size_t)g * scale_stride + blockIdx.x] = s;
      s_scale[g] = fp8_scale(s);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int j = at(i), g = (j + off) / 128;  // the group of all its elements but, in the first, `off` of them
      if (j >= H) continue;
      const Fp8Scale f = s_scale[min(g, G - 1)], f0 = (j + off) % 128 == 0 ? s_scale[max(g - 1, 0)] : f;
      uint32_t w[N / 4];
#pragma unroll
      for (int k = 0; k < N; ++k) {
        const Fp8Scale fk = k < off ? f0 : f;
        n[i][k] = n[i][k] * fk.up * fk.inv;
      }
      make_codes<N>(w, n[i]);
      if (whole(j)) {
        store_codes<N>(codes + row + j, w);
      } else {
#pragma unroll
        for (int k = 0; k < N; ++k)
          if (inside(j, k)) codes[row + j + k] = (uint8_t)(w[k / 4] >> (8 * (k % 4)));
      }
    }
  }
}

template <typename T>
using NormKernel = void (*)(int, const T*, const T*, const T*, float, T*, T*, uint8_t*, float*, int64_t);

template <typename T, bool SHIFT>
NormKernel<T> vec_kernel(int nv) {
  return nv == 1   ? add_rmsnorm_vec_kernel<T, 1, SHIFT>
         : nv == 2 ? add_rmsnorm_vec_kernel<T, 2, SHIFT>
                   : add_rmsnorm_vec_kernel<T, 4, SHIFT>;
}

template <typename T>
fp4moe_status norm_launch(int32_t rows, int32_t H, const void* x, const void* residual, const void* gamma, float eps,
                          void* h_out, void* y, uint8_t* codes, float* scales, int64_t scale_stride,
                          cudaStream_t st) {
  constexpr int N = 16 / (int)sizeof(T);
  NormKernel<T> kernel = add_rmsnorm_any_kernel<T>;
  int threads = NORM_THREADS;
  const int nsm = sm_count();
  if (nsm <= 0) return FP4MOE_CUDA_ERROR;
  const bool shift = H % N != 0;
  // vectors of a row: one more where its first element lies inside a vector
  const int64_t vecs = shift ? ((int64_t)H + 2 * N - 2) / N : H / N;
  if (vecs <= 4 * 1024) {
    // vectors a thread: one while the rows leave SMs idle, then two, and as many as 1024 threads need
    int nv = rows <= nsm ? 1 : 2;
    while ((vecs + nv - 1) / nv > 1024) nv *= 2;
    threads = (int)((vecs + nv - 1) / nv + 31) / 32 * 32;
    kernel = shift ? vec_kernel<T, true>(nv) : vec_kernel<T, false>(nv);
  }
  const cudaError_t r =
      launch_pdl(kernel, dim3((unsigned)rows), dim3((unsigned)threads), 0, st, H, static_cast<const T*>(x),
                 static_cast<const T*>(residual), static_cast<const T*>(gamma), eps, static_cast<T*>(h_out),
                 static_cast<T*>(y), codes, scales, scale_stride);
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
