// Microscaled 4-bit quantisation of a plain matrix, and its inverse.
//
// A row of K elements is cut into blocks of 32 (MXFP4, E8M0 scales) or 16 (NVFP4, E4M3 scales under a global
// scale g); the last block may be short, and counts as if zeros followed. Per block, in IEEE fp32 with RNE:
//   MXFP4 (OCP Microscaling v1.0)   X = floor(log2 a) - 2 clamped to [-127, 127], -127 where a == 0;
//                                   scale byte X + 127, code E2M1_satfinite(v * 2^-X)
//   NVFP4                           quant_block16 (common.cuh)
// where a = max|v|. A block that holds an infinity or a NaN gets the NaN scale (0xFF, 0x7F) and zero codes, so
// whatever is computed from it is NaN rather than a plausible number.
// Codes: row r at r * ceil(K / 32) * 16 bytes, element 2i in the low nibble of byte i, zero past K. Scales in
// 128 x 4 tiles (sf_offset, common.cuh), zero in the rows and columns that only fill a tile: a tensor-core
// product may read those, and a zero scale byte is a finite scale in either format.
#include "common.cuh"
#include "dense.cuh"
#include "internal.h"

namespace fp4moe {
namespace {

constexpr int MQ_THREADS = 256;

// 2^-X for X in [-127, 125]
__device__ __forceinline__ float exp2_neg(int X) { return __uint_as_float((uint32_t)(127 - X) << 23); }

// One block of 16 elements: the code bytes and the scale byte. MXFP4 joins the amax of two lanes.
template <int FMT>
__device__ __forceinline__ uint32_t quantize16(const float (&v)[16], float g, uint32_t& lo, uint32_t& hi) {
  float a = 0.0f;
#pragma unroll
  for (int i = 0; i < 16; ++i) a = fmax_nan(a, fabsf(v[i]));
  if constexpr (FMT == FP4MOE_W_MXFP4) a = fmax_nan(a, __shfl_xor_sync(0xFFFFFFFFu, a, 1));
  const bool bad = !(a <= 3.402823466e38f);
  uint32_t sf;
  if constexpr (FMT == FP4MOE_W_MXFP4) {
    // floor(log2 a) of a normal a is its biased exponent - 127. A subnormal a lies below 2^-126, so its X
    // clamps at -127 as the biased exponent 0 does.
    const int X = bad ? 0 : max((int)(__float_as_uint(a) >> 23) - 129, -127);
    const float inv = exp2_neg(X);
    lo = hi = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) lo |= cvt_e2m1x2(v[2 * i] * inv, v[2 * i + 1] * inv) << (8 * i);
#pragma unroll
    for (int i = 0; i < 4; ++i) hi |= cvt_e2m1x2(v[8 + 2 * i] * inv, v[9 + 2 * i] * inv) << (8 * i);
    sf = bad ? 0xFFu : (uint32_t)(X + 127);
  } else {
    sf = quant_block16(v, g, lo, hi);
    if (bad) sf = 0x7Fu;
  }
  if (bad) lo = hi = 0;
  return sf;
}

// A thread takes pieces of 16 elements. Rows are padded to whole 128s and columns to whole scale tiles, so that
// every byte of the scale tiles is written. Pieces of a padded row come in multiples of four, so both halves of
// a 32-element block sit in neighbouring lanes, and a warp is inside or past the last piece as a whole.
template <int FMT, typename T>
__global__ void __launch_bounds__(MQ_THREADS)
    mx_quantize_any_kernel(int rows, int K, int64_t pieces, int segs, int col_tiles, int64_t row_bytes,
                           const T* __restrict__ x, const float* __restrict__ gs, uint8_t* __restrict__ codes,
                           uint8_t* __restrict__ sf_out) {
  constexpr int B = MxFormat<FMT>::kBlock;
  pdl_wait();
  pdl_trigger();
  const float g = FMT == FP4MOE_W_NVFP4 ? __ldg(gs) : 1.0f;
  for (int64_t i = (int64_t)blockIdx.x * MQ_THREADS + threadIdx.x; i < pieces; i += (int64_t)gridDim.x * MQ_THREADS) {
    const int64_t r = i / segs;
    const int seg = (int)(i - r * segs);
    float v[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const int64_t k = (int64_t)seg * 16 + j;
      v[j] = (r < rows && k < K) ? to_f32(x[(size_t)r * K + k]) : 0.0f;
    }
    uint32_t lo, hi;
    uint32_t sf = quantize16<FMT>(v, g, lo, hi);
    if (r < rows && (int64_t)seg * 8 < row_bytes)
      *reinterpret_cast<uint2*>(codes + (size_t)r * row_bytes + (size_t)seg * 8) = make_uint2(lo, hi);
    const int c = seg * 16 / B;
    if (r >= rows || (int64_t)c * B >= K) sf = 0;
    if (B == 16 || (seg & 1) == 0) sf_out[mx_sf_offset((uint64_t)r, (uint32_t)c, (uint64_t)col_tiles)] = (uint8_t)sf;
  }
}

// value = e2m1(code) * scale, divided by g (NVFP4), rounded once.
template <int FMT, typename T>
__global__ void __launch_bounds__(MQ_THREADS)
    mx_dequantize_any_kernel(int rows, int K, int col_tiles, int64_t row_bytes, const uint8_t* __restrict__ codes,
                             const uint8_t* __restrict__ sf, const float* __restrict__ gs, T* __restrict__ out) {
  constexpr int B = MxFormat<FMT>::kBlock;
  pdl_wait();
  pdl_trigger();
  const float g = FMT == FP4MOE_W_NVFP4 ? __ldg(gs) : 1.0f;
  const int64_t n = (int64_t)rows * K;
  for (int64_t i = (int64_t)blockIdx.x * MQ_THREADS + threadIdx.x; i < n; i += (int64_t)gridDim.x * MQ_THREADS) {
    const int64_t r = i / K;
    const int k = (int)(i - r * K);
    const uint32_t q = (uint32_t)codes[(size_t)r * row_bytes + k / 2] >> (4 * (k & 1)) & 15u;
    const float s = mx_scale<FMT>(sf[mx_sf_offset((uint64_t)r, (uint32_t)(k / B), (uint64_t)col_tiles)]);
    float v = e2m1_to_f32(q) * s;
    if (FMT == FP4MOE_W_NVFP4) v = __fdiv_rn(v, g);
    out[i] = from_f32<T>(v);
  }
}

// CTAs of a grid-stride loop over n items of MQ_THREADS each: enough to fill the device several times over.
unsigned stride_grid(int64_t n) {
  const int64_t want = (n + MQ_THREADS - 1) / MQ_THREADS, most = (int64_t)sm_count() * 32;
  return (unsigned)(want < most ? want : most);
}

template <int FMT, typename T>
fp4moe_status quantize_launch(int32_t rows, int32_t K, const void* x, const float* gs, uint8_t* codes, uint8_t* sf,
                              cudaStream_t st) {
  const int64_t ct = mx_col_tiles(FMT, K), segs = ct * 4 * MxFormat<FMT>::kBlock / 16;
  const int64_t pieces = mx_row_tiles(rows) * 128 * segs;
  return launch_pdl(mx_quantize_any_kernel<FMT, T>, dim3(stride_grid(pieces)), dim3(MQ_THREADS), 0, st, rows, K,
                    pieces, (int)segs, (int)ct, mx_row_bytes(K), static_cast<const T*>(x), gs, codes,
                    sf) == cudaSuccess
             ? FP4MOE_OK
             : FP4MOE_CUDA_ERROR;
}

template <int FMT, typename T>
fp4moe_status dequantize_launch(int32_t rows, int32_t K, const uint8_t* codes, const uint8_t* sf, const float* gs,
                                void* out, cudaStream_t st) {
  return launch_pdl(mx_dequantize_any_kernel<FMT, T>, dim3(stride_grid((int64_t)rows * K)), dim3(MQ_THREADS), 0, st,
                    rows, K, (int)mx_col_tiles(FMT, K), mx_row_bytes(K), codes, sf, gs,
                    static_cast<T*>(out)) == cudaSuccess
             ? FP4MOE_OK
             : FP4MOE_CUDA_ERROR;
}

}  // namespace

fp4moe_status mx_quantize_launch(int32_t format, int32_t dtype, int32_t rows, int32_t K, const void* x,
                                 const float* gs, uint8_t* codes, uint8_t* sf, cudaStream_t st) {
  if (sm_count() <= 0) return FP4MOE_CUDA_ERROR;
  constexpr int NV = FP4MOE_W_NVFP4, MX = FP4MOE_W_MXFP4;
  if (format == MX) {
    if (dtype == FP4MOE_BF16) return quantize_launch<MX, __nv_bfloat16>(rows, K, x, gs, codes, sf, st);
    if (dtype == FP4MOE_FP16) return quantize_launch<MX, __half>(rows, K, x, gs, codes, sf, st);
    return quantize_launch<MX, float>(rows, K, x, gs, codes, sf, st);
  }
  if (dtype == FP4MOE_BF16) return quantize_launch<NV, __nv_bfloat16>(rows, K, x, gs, codes, sf, st);
  if (dtype == FP4MOE_FP16) return quantize_launch<NV, __half>(rows, K, x, gs, codes, sf, st);
  return quantize_launch<NV, float>(rows, K, x, gs, codes, sf, st);
}

fp4moe_status mx_dequantize_launch(int32_t format, int32_t dtype, int32_t rows, int32_t K, const uint8_t* codes,
                                   const uint8_t* sf, const float* gs, void* out, cudaStream_t st) {
  if (sm_count() <= 0) return FP4MOE_CUDA_ERROR;
  constexpr int NV = FP4MOE_W_NVFP4, MX = FP4MOE_W_MXFP4;
  if (format == MX) {
    if (dtype == FP4MOE_BF16) return dequantize_launch<MX, __nv_bfloat16>(rows, K, codes, sf, gs, out, st);
    if (dtype == FP4MOE_FP16) return dequantize_launch<MX, __half>(rows, K, codes, sf, gs, out, st);
    return dequantize_launch<MX, float>(rows, K, codes, sf, gs, out, st);
  }
  if (dtype == FP4MOE_BF16) return dequantize_launch<NV, __nv_bfloat16>(rows, K, codes, sf, gs, out, st);
  if (dtype == FP4MOE_FP16) return dequantize_launch<NV, __half>(rows, K, codes, sf, gs, out, st);
  return dequantize_launch<NV, float>(rows, K, codes, sf, gs, out, st);
}

}  // namespace fp4moe
