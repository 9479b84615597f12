// Residual addition and root-mean-square norm, with an optional block-FP8 copy of the result.
//
//   h[t]  = RN(x[t] + residual[t])                    (the stored residual stream; h = x without a residual)
//   n[t]  = h[t] * rsqrt(mean_j h[t, j]^2 + eps) * gamma
//   y[t]  = RN(n[t]),   s[t, g] = amax_g |n| / 448,   code = E4M3_satfinite(n / s), 0 where s == 0
// for the 1 x 128 groups g of a row: the activation format of the block-FP8 shared expert (segemm.cu). The
// codes are not taken from the y that was rounded to its type, so they carry one rounding, not two. n has one order of
// products, (h rstd) gamma, in every kernel, with and without the codes; these come from h gamma (Fp8Ratio).
//
// The sum of squares and the statistics are fp32; h is rounded to its storage type first, so the norm is
// that of the stream a later layer reads back.
//
// Bound by memory: a row is read and written once. One CTA takes a row and, where it fits, keeps it in registers
// between the two uses. Few rows leave the device empty and the time is one trip to memory, a reduction and a trip
// back (1 x 4096 bf16 2.0 us, 64 rows 2.3 us), so they take the most threads; many rows take two or four 16-byte
// vectors a thread (8192 x 4096 bf16 with the FP8 copy 48.6 us, 6.2 TB/s, 92 % of a copy's rate).
#include "common.cuh"
#include "dense.cuh"
#include "internal.h"

namespace fp4moe {
namespace {

constexpr int NORM_THREADS = 1024;

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

// The largest of 32 lanes, NaN if any is, in every lane.
__device__ __forceinline__ float warp_max_nan(float v) {
  float r;
  asm volatile("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}

// The codes of a group are RN_E4M3(v / t), v and t being n and s up to one factor. The quotient is off by half a unit
// of fp32's last place in all but rare cases: one reciprocal serves a group, and two fused steps per element take its
// error out.
struct Fp8Ratio {
  float t, inv;
};
__device__ __forceinline__ float fp8_quotient(float v, const Fp8Ratio& f) {
  const float q = v * f.inv;
  return fmaf(fmaf(-q, f.t, v), f.inv, q);
}
// rstd is a factor of n and s, so it is left out: v = 448 p with p = h * gamma, t = amax|p|. In bf16 these are exact
// in fp32 (19 and 16 bits), so quotients that lie on a tie between two E4M3 values stay on it, no others come as near
// as the last rounding, and the codes are those of exact arithmetic. (fp16: v has one rounding at most; fp32: p and v
// each.) n, amax and s would bring six roundings. Needs p, rstd and their products well inside fp32's range.
__device__ __forceinline__ bool in_range(float v) { return v > 0x1p-50f && v < 0x1p50f; }
__device__ __forceinline__ Fp8Ratio fp8_ratio(float a) { return Fp8Ratio{a, __frcp_rn(a)}; }
// Any other group: v = n * up, t = s * up; 0 where s == 0. Below 2^-120 the reciprocal would overflow, so n and s are
// first scaled up by 2^100, exactly (a subnormal n included). s = inf: finite n give 0, infinite ones NaN.
__device__ __forceinline__ Fp8Ratio fp8_scale(float s, float& up) {
  up = s == 0.0f ? 0.0f : s < 0x1p-120f ? 0x1p100f : 1.0f;
  const float t = s * (s < 0x1p-120f ? 0x1p100f : 1.0f);
  return Fp8Ratio{isinf(s) ? 0.0f : t, s == 0.0f ? 0.0f : __frcp_rn(t)};
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

// Widths too large for a CTA's registers: element accesses, and the row is read again for its second use
// (500 x 40960 bf16 with the FP8 copy 74 us, 2.5 TB/s; with 256 threads 111 us). A warp takes whole 128-element
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
    float n[4], p[4], a = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int j = g * 128 + 32 * i + lane;
      n[i] = p[i] = 0.0f;
      if (j < H) {
        float h = to_f32(x[row + j]);
        if (residual != nullptr) {
          const T r = from_f32<T>(__fadd_rn(h, to_f32(residual[row + j])));
          h = to_f32(r);
          h_out[row + j] = r;
        }
        const float w = gamma != nullptr ? to_f32(gamma[j]) : 1.0f;
        n[i] = h * rstd * w;
        p[i] = h * w;
        if (y != nullptr) y[row + j] = from_f32<T>(n[i]);
      }
      a = fmax_nan(a, fabsf(p[i]));
    }
    if (codes != nullptr) {
      a = warp_max_nan(a);
      float s;
      Fp8Ratio f;
      if (in_range(a) && in_range(rstd)) {
        f = fp8_ratio(a);
        s = __fdiv_rn(a, 448.0f) * rstd;
#pragma unroll
        for (int i = 0; i < 4; ++i) p[i] *= 448.0f;
      } else {
        a = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) a = fmax_nan(a, fabsf(n[i]));
        s = __fdiv_rn(warp_max_nan(a), 448.0f);  // a NaN takes its whole group along: NaN scale, NaN codes
        float up;
        f = fp8_scale(s, up);
#pragma unroll
        for (int i = 0; i < 4; ++i) p[i] = n[i] * up;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int j = g * 128 + 32 * i + lane;
        if (j < H) codes[row + j] = (uint8_t)cvt_e4m3x2(fp8_quotient(p[i], f), 0.0f);
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

// Widths that 16-byte vectors divide. Vector q of a row, in a thread's slot i, is q = i * blockDim + threadIdx; the
// vectors of one FP8 group are 128 / N neighbouring lanes.
template <typename T, int NV>
__global__ void __launch_bounds__(1024)
    add_rmsnorm_vec_kernel(int H, const T* x, const T* residual, const T* __restrict__ gamma, float eps, T* h_out,
                           T* y, uint8_t* codes, float* scales, int64_t scale_stride) {
  constexpr int N = 16 / (int)sizeof(T), LANES = 128 / N;
  static_assert(LANES == 16 || LANES == 32, "a group is a warp or half of one");
  __shared__ float s_red[32];
  pdl_wait();
  pdl_trigger();
  const size_t row = (size_t)blockIdx.x * H;
  auto at = [&](int i) { return (i * (int)blockDim.x + (int)threadIdx.x) * N; };
  // Every load of the row is issued before the first is waited for. gamma waits until x and the residual are joined
  // where its registers would cost occupancy (8192 x 4096 bf16, the norm alone, two vectors: 27 against 30 us).
  uint4 hv[NV], rv[NV], gv[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int j = at(i);
    hv[i] = rv[i] = gv[i] = make_uint4(0, 0, 0, 0);
    if (j < H) {
      hv[i] = ld_vec(x + row + j);
      if (residual != nullptr) rv[i] = ld_vec(residual + row + j);
      if (NV == 1 && gamma != nullptr) gv[i] = __ldg(reinterpret_cast<const uint4*>(gamma + j));
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
      if (at(i) < H) *reinterpret_cast<uint4*>(h_out + row + at(i)) = hv[i];
    }
  }
  if constexpr (NV > 1) {
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
  auto group_max = [](float a, uint32_t lanes) {
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) a = fmax_nan(a, __shfl_xor_sync(lanes, a, o));
    return a;
  };
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int j = at(i);
    float p[N], g[N], n[N];
    unpack<T>(hv[i], p);
    unpack<T>(gv[i], g);
    auto norm = [&]() {  // one order of the products, whether or not there are codes
      float h[N];
      unpack<T>(hv[i], h);
#pragma unroll
      for (int k = 0; k < N; ++k) n[k] = gamma != nullptr ? h[k] * rstd * g[k] : h[k] * rstd;
    };
    if (codes == nullptr) {
      norm();
      if (j < H) *reinterpret_cast<uint4*>(y + row + j) = pack<T>(n);
      continue;
    }
    float a = 0.0f, s;
#pragma unroll
    for (int k = 0; k < N; ++k) {
      if (gamma != nullptr) p[k] *= g[k];
      a = fmax_nan(a, fabsf(p[k]));
    }
    a = group_max(a, 0xFFFFFFFFu);
    norm();
    Fp8Ratio f;
    if (in_range(a) && in_range(rstd)) {
      f = fp8_ratio(a);
      s = __fdiv_rn(a, 448.0f) * rstd;
#pragma unroll
      for (int k = 0; k < N; ++k) p[k] *= 448.0f;
    } else {
      a = 0.0f;
#pragma unroll
      for (int k = 0; k < N; ++k) a = fmax_nan(a, fabsf(n[k]));  // a NaN takes its whole group along
      // the way to the codes is the group's own: the warp's other group may have gone the short one
      const uint32_t mates = LANES == 32 ? 0xFFFFFFFFu : 0xFFFFu << (threadIdx.x & 16u);
      s = __fdiv_rn(group_max(a, mates), 448.0f);
      float up;
      f = fp8_scale(s, up);
#pragma unroll
      for (int k = 0; k < N; ++k) p[k] = n[k] * up;
    }
    if (j >= H) continue;
    if (y != nullptr) *reinterpret_cast<uint4*>(y + row + j) = pack<T>(n);
#pragma unroll
    for (int k = 0; k < N; ++k) n[k] = fp8_quotient(p[k], f);
    uint32_t w[N / 4];
    make_codes<N>(w, n);
    store_codes<N>(codes + row + j, w);
    if (j % 128 == 0) scales[(size_t)(j / 128) * scale_stride + blockIdx.x] = s;
  }
}

// U elements of a row in one access of U * sizeof(T) bytes: 2, 4 or 8.
template <typename T, int U>
using Raw = std::conditional_t<U * sizeof(T) == 2, uint16_t, std::conditional_t<U * sizeof(T) == 4, uint32_t, uint2>>;
template <typename T, int U>
__device__ __forceinline__ void unpack_raw(Raw<T, U> q, float (&v)[U]) {
  if constexpr (U == 1) {
    v[0] = to_f32(*reinterpret_cast<const T*>(&q));
  } else {
    uint4 w = make_uint4(0, 0, 0, 0);
    if constexpr (sizeof(q) == 4) {
      w.x = q;
    } else {
      w.x = q.x;
      w.y = q.y;
    }
    float f[16 / sizeof(T)];
    unpack<T>(w, f);
#pragma unroll
    for (int k = 0; k < U; ++k) v[k] = f[k];
  }
}
template <typename T, int U>
__device__ __forceinline__ Raw<T, U> pack_raw(const float (&v)[U]) {
  if constexpr (U == 1) {
    const T t = from_f32<T>(v[0]);
    return *reinterpret_cast<const Raw<T, 1>*>(&t);
  } else if constexpr (sizeof(T) == 4) {
    return make_uint2(__float_as_uint(v[0]), __float_as_uint(v[1]));
  } else if constexpr (U == 2) {
    return pack2<T>(v[0], v[1]);
  } else {
    return make_uint2(pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3]));
  }
}

// Widths that the 16-byte vectors do not divide. Rows then start at any element, and a vector that is aligned for
// one row is not for the next, so a lane reads and writes U elements at a time, the most that divide H (4, 2 or
// 1), in accesses that are contiguous over the warp. A warp takes whole FP8 groups: NG of them, in registers, and
// a group's maximum is one warp reduction. 8192 x 4090 bf16 with the FP8 copy 57 us, 8192 x 4092 53 us, 8192 x 4095
// (single elements: bound by the accesses) 82 us, against 77, 75 and 78 us with whole vectors that were cut at the
// aligned addresses and shifted into place, and 49 us at 4096. 1000 x 4090 fp16: 8.9 against 12.2 us.
template <typename T, int U, int NG>
__global__ void __launch_bounds__(1024)
    add_rmsnorm_group_kernel(int H, const T* x, const T* residual, const T* __restrict__ gamma, float eps, T* h_out,
                             T* y, uint8_t* codes, float* scales, int64_t scale_stride) {
  constexpr int S = 4 / U;
  using R = Raw<T, U>;
  __shared__ float s_red[32];
  pdl_wait();
  pdl_trigger();
  const size_t row = (size_t)blockIdx.x * H;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  auto at = [&](int i, int s) { return (i * warps + warp) * 128 + (s * 32 + lane) * U; };
  R hv[NG][S], rv[NG][S], gv[NG][S];
#pragma unroll
  for (int i = 0; i < NG; ++i)
#pragma unroll
    for (int s = 0; s < S; ++s) {
      const int j = at(i, s);
      hv[i][s] = rv[i][s] = gv[i][s] = R{};
      if (j < H) {
        hv[i][s] = *reinterpret_cast<const R*>(x + row + j);
        if (residual != nullptr) rv[i][s] = *reinterpret_cast<const R*>(residual + row + j);
        if (NG == 1 && gamma != nullptr) gv[i][s] = __ldg(reinterpret_cast<const R*>(gamma + j));
      }
    }
  float ss = 0.0f;
#pragma unroll
  for (int i = 0; i < NG; ++i)
#pragma unroll
    for (int s = 0; s < S; ++s) {
      const int j = at(i, s);
      float h[U], r[U];
      unpack_raw<T, U>(hv[i][s], h);
      if (residual != nullptr) {
        unpack_raw<T, U>(rv[i][s], r);
#pragma unroll
        for (int k = 0; k < U; ++k) h[k] = __fadd_rn(h[k], r[k]);
        hv[i][s] = pack_raw<T, U>(h);
        if (j < H) *reinterpret_cast<R*>(h_out + row + j) = hv[i][s];
        unpack_raw<T, U>(hv[i][s], h);
      }
#pragma unroll
      for (int k = 0; k < U; ++k) ss = fmaf(h[k], h[k], ss);
    }
  if constexpr (NG > 1) {  // with several groups gamma takes the residual's registers
#pragma unroll
    for (int i = 0; i < NG; ++i)
#pragma unroll
      for (int s = 0; s < S; ++s)
        if (gamma != nullptr && at(i, s) < H) gv[i][s] = __ldg(reinterpret_cast<const R*>(gamma + at(i, s)));
  }
  ss = cta_sum(ss, s_red);
  const float rstd = __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(__fdiv_rn(ss, (float)H), eps)));
#pragma unroll
  for (int i = 0; i < NG; ++i) {
    const int g = i * warps + warp;
    if (g * 128 >= H) break;
    float n[S][U], p[S][U], w[S][U];
#pragma unroll
    for (int s = 0; s < S; ++s) {
      unpack_raw<T, U>(hv[i][s], p[s]);
      unpack_raw<T, U>(gv[i][s], w[s]);
    }
    auto norm = [&]() {  // one order of the products, whether or not there are codes
      float h[S][U];
#pragma unroll
      for (int s = 0; s < S; ++s) unpack_raw<T, U>(hv[i][s], h[s]);
#pragma unroll
      for (int s = 0; s < S; ++s)
#pragma unroll
        for (int k = 0; k < U; ++k) n[s][k] = gamma != nullptr ? h[s][k] * rstd * w[s][k] : h[s][k] * rstd;
    };
    float a = 0.0f, sc = 0.0f;
    Fp8Ratio f{};
    norm();
    if (codes != nullptr) {
#pragma unroll
      for (int s = 0; s < S; ++s)
#pragma unroll
        for (int k = 0; k < U; ++k) {
          if (gamma != nullptr) p[s][k] *= w[s][k];
          a = fmax_nan(a, fabsf(p[s][k]));
        }
      a = warp_max_nan(a);
      if (in_range(a) && in_range(rstd)) {
        f = fp8_ratio(a);
        sc = __fdiv_rn(a, 448.0f) * rstd;
#pragma unroll
        for (int s = 0; s < S; ++s)
#pragma unroll
          for (int k = 0; k < U; ++k) p[s][k] *= 448.0f;
      } else {
        a = 0.0f;
#pragma unroll
        for (int s = 0; s < S; ++s)
#pragma unroll
          for (int k = 0; k < U; ++k) a = fmax_nan(a, fabsf(n[s][k]));
        sc = __fdiv_rn(warp_max_nan(a), 448.0f);  // a NaN takes its whole group along
        float up;
        f = fp8_scale(sc, up);
#pragma unroll
        for (int s = 0; s < S; ++s)
#pragma unroll
          for (int k = 0; k < U; ++k) p[s][k] = n[s][k] * up;
      }
    }
#pragma unroll
    for (int s = 0; s < S; ++s) {
      const int j = at(i, s);
      if (j >= H) continue;
      if (y != nullptr) *reinterpret_cast<R*>(y + row + j) = pack_raw<T, U>(n[s]);
      if (codes == nullptr) continue;
#pragma unroll
      for (int k = 0; k < U; ++k) n[s][k] = fp8_quotient(p[s][k], f);
      if constexpr (U == 4) {
        uint32_t w[1];
        make_codes<4>(w, n[s]);
        *reinterpret_cast<uint32_t*>(codes + row + j) = w[0];
      } else if constexpr (U == 2) {
        *reinterpret_cast<uint16_t*>(codes + row + j) = (uint16_t)cvt_e4m3x2(n[s][0], n[s][1]);
      } else {
        codes[row + j] = (uint8_t)cvt_e4m3x2(n[s][0], 0.0f);
      }
    }
    if (codes != nullptr && lane == 0) scales[(size_t)g * scale_stride + blockIdx.x] = sc;
  }
}

template <typename T>
using NormKernel = void (*)(int, const T*, const T*, const T*, float, T*, T*, uint8_t*, float*, int64_t);

template <typename T>
NormKernel<T> vec_kernel(int nv) {
  return nv == 1   ? add_rmsnorm_vec_kernel<T, 1>
         : nv == 2 ? add_rmsnorm_vec_kernel<T, 2>
                   : add_rmsnorm_vec_kernel<T, 4>;
}
template <typename T, int U>
NormKernel<T> group_kernel(int ng) {
  if constexpr (sizeof(T) == 2 && U > 1)
    if (ng == 8) return add_rmsnorm_group_kernel<T, U, 8>;
  return ng == 1 ? add_rmsnorm_group_kernel<T, U, 1> : add_rmsnorm_group_kernel<T, U, 4>;
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
  const int64_t vecs = ((int64_t)H + N - 1) / N, groups = ((int64_t)H + 127) / 128;
  if (H % N == 0 && vecs <= 4 * 1024) {
    // vectors a thread: one while the rows leave SMs idle, two while an SM has one row or two or a row leaves four
    // warps idle, else four, and as many as 1024 threads need (bf16 with the FP8 copy, two and four: 300 x 4096 3.0
    // and 3.6 us, 8192 x 2048 25.4 and 26.4, 8192 x 4096 50.8 and 48.5, 4096 x 7168 50.4 and 43.7, 2000 x 8192 28.5
    // and 26.5)
    int nv = rows <= nsm ? 1 : rows <= 2 * nsm || vecs < 512 ? 2 : 4;
    while ((vecs + nv - 1) / nv > 1024) nv *= 2;
    threads = (int)((vecs + nv - 1) / nv + 31) / 32 * 32;
    kernel = vec_kernel<T>(nv);
  } else if (H % N != 0 && groups <= (sizeof(T) == 2 && H % 2 == 0 ? 8 : 4) * 32) {
    // groups a warp: one while the rows leave SMs idle (64 x 4090 bf16 2.7 us, with eight 4.7), then four (8192 x 4090
    // 57 us; one 96, eight 62), and eight where 32 warps need them and their registers suffice
    const int ng = groups > 4 * 32 ? 8 : rows > nsm || groups > 32 ? 4 : 1;
    threads = (int)((groups + ng - 1) / ng) * 32;
    if constexpr (sizeof(T) == 4)
      kernel = H % 2 == 0 ? group_kernel<T, 2>(ng) : group_kernel<T, 1>(ng);
    else
      kernel = H % 4 == 0 ? group_kernel<T, 4>(ng) : H % 2 == 0 ? group_kernel<T, 2>(ng) : group_kernel<T, 1>(ng);
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
