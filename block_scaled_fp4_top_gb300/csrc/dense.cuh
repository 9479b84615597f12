// Element types and 4-bit block formats of the dense operators (norm.cu, mxquant.cu, mxdense.cu).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "common.cuh"

namespace fp4moe {

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }

// One rounding to nearest even into the storage type.
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }

// 16 bytes of T as fp32 values, and back with one rounding each.
template <typename T>
__device__ __forceinline__ void unpack(uint4 q, float (&v)[16 / sizeof(T)]) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(T) == 4) {
      v[i] = __uint_as_float(w[i]);
    } else if constexpr (std::is_same_v<T, __nv_bfloat16>) {
      v[2 * i] = bf16_lo(w[i]);
      v[2 * i + 1] = bf16_hi(w[i]);
    } else {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    }
  }
}
template <typename T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if constexpr (std::is_same_v<T, __nv_bfloat16>) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&p);
  } else {
    const __half2 p = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&p);
  }
}
template <typename T>
__device__ __forceinline__ uint4 pack(const float (&v)[16 / sizeof(T)]) {
  if constexpr (sizeof(T) == 4)
    return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
  else
    return make_uint4(pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3]), pack2<T>(v[4], v[5]), pack2<T>(v[6], v[7]));
}

// The OUT words from byte `drop` on of the IN words w, in place: drop is even and less than 16.
template <int IN, int OUT>
__device__ __forceinline__ void shift_words(uint32_t (&w)[IN], int drop) {
  static_assert(IN >= OUT + 4, "16 - 2 bytes can be dropped");
#pragma unroll
  for (int i = 0; i < OUT + 2; ++i) w[i] = (drop & 8) ? w[i + 2] : w[i];
#pragma unroll
  for (int i = 0; i < OUT + 1; ++i) w[i] = (drop & 4) ? w[i + 1] : w[i];
  const uint32_t sel = (drop & 2) ? 0x5432u : 0x3210u;
#pragma unroll
  for (int i = 0; i < OUT; ++i) w[i] = __byte_perm(w[i], w[i + 1], sel);
}

// 32 bytes at a 32-byte-aligned address in one access (256-bit, sm_100 and later): a thread fills whole sectors.
__device__ __forceinline__ void ld_global_32(const void* p, uint4& a, uint4& b) {
  asm volatile("ld.global.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(a.x), "=r"(a.y), "=r"(a.z), "=r"(a.w), "=r"(b.x), "=r"(b.y), "=r"(b.z), "=r"(b.w)
               : "l"(p));
}
__device__ __forceinline__ void st_global_32(void* p, uint4 a, uint4 b) {
  asm volatile("st.global.L1::no_allocate.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(a.x), "r"(a.y),
               "r"(a.z), "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
               : "memory");
}

// Two signed E4M3 codes (RNE, satfinite; NaN gives the NaN code): `lo` in the low byte.
__device__ __forceinline__ uint32_t cvt_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// The value of an E2M1 code: 0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives.
__device__ __forceinline__ float e2m1_to_f32(uint32_t q) {
  const uint32_t e = (q >> 1) & 3u, m = q & 1u;
  const float v = e ? __uint_as_float(((e + 126u) << 23) | (m << 22)) : 0.5f * (float)m;
  return (q & 8u) ? -v : v;
}

// The microscaled 4-bit formats: elements per scale.
template <int FMT>
struct MxFormat;
template <>
struct MxFormat<FP4MOE_W_NVFP4> {
  static constexpr int kBlock = 16;
};
template <>
struct MxFormat<FP4MOE_W_MXFP4> {
  static constexpr int kBlock = 32;
};

// The value of a scale byte: E8M0 is 2^(b - 127) with 0xFF for NaN; E4M3 has NaN at 0x7F.
template <int FMT>
__device__ __forceinline__ float mx_scale(uint32_t b) {
  if constexpr (FMT == FP4MOE_W_MXFP4)
    return b == 255u ? __uint_as_float(0x7FC00000u) : (b == 0u ? 0x1p-127f : __uint_as_float(b << 23));
  else
    return b == 0x7Fu ? __uint_as_float(0x7FC00000u) : e4m3_to_f32(b);
}

// sf_offset for matrices of any size: byte offset of scale (r, c), with col_tiles tiles across.
__device__ __forceinline__ size_t mx_sf_offset(uint64_t r, uint32_t c, uint64_t col_tiles) {
  return (size_t)(((r >> 7) * col_tiles + (c >> 2)) * 512u + (r & 31u) * 16u + ((r & 127u) >> 5) * 4u + (c & 3u));
}

inline int mx_block(int32_t format) { return format == FP4MOE_W_MXFP4 ? 32 : 16; }
// Bytes of one row of codes: K rounded up to whole 32-element groups, so that every row starts 16-byte aligned.
inline int64_t mx_row_bytes(int32_t K) { return ((int64_t)K + 31) / 32 * 16; }
// 128 x 4 scale tiles of a matrix: row tiles and column tiles.
inline int64_t mx_row_tiles(int32_t rows) { return ((int64_t)rows + 127) / 128; }
inline int64_t mx_col_tiles(int32_t format, int32_t K) {
  const int64_t b = mx_block(format);
  return (((int64_t)K + b - 1) / b + 3) / 4;
}

}  // namespace fp4moe
