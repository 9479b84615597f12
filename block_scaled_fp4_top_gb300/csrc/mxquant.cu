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
//
// Both directions are bound by memory: 8192 x 4096 bf16 is 84 MB in and out, 12.4 us at the copy rate, and takes
// 15.5 us to MXFP4 and 16.4 to NVFP4, 14.9 and 16.2 us back. A thread takes 32 bytes of the plain matrix, one whole
// sector, in one 256-bit access where rows are 32-byte aligned (two 16-byte ones: 19.5 us). Rows at any other
// element are read and written in aligned vectors too, shifted into place in registers (8192 x 4095: 20 and 23 us).
#include <algorithm>

#include "common.cuh"
#include "dense.cuh"
#include "internal.h"

namespace fp4moe {
namespace {

constexpr int MQ_THREADS = 256;
// More rows than this many CTAs an SM take are looped over, with the next row's loads in flight: 8192 x 4096 bf16 to
// MXFP4 takes 15.5 us with 8, 15.6 with 4, 15.9 with 12 and 21.5 without a loop; the inverse, whose CTAs hold fewer
// registers, 15.4, 15.8, 14.9 and 16.5.
constexpr int kCtasPerSm = 8, kCtasPerSmInverse = 12;

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

// 16 elements of T from element e of a buffer of n elements: aligned 16-byte loads, shifted into place where e
// lies inside a vector. Vectors that reach past the buffer are read element by element (zeros past it); vectors
// that hold a neighbour row's elements are not, those are only dropped. The loads and their use are apart, so
// that a row's loads are in flight while the row before is worked on.
// WIDE: every piece starts 32-byte aligned and lies inside the buffer or past it, so 256-bit loads reach it.
template <typename T, bool WIDE>
struct Piece16 {
  static constexpr int N = 16 / (int)sizeof(T), W = 16 / N;  // elements a vector, vectors wanted
  uint4 q[W + 1];
  int off;
  __device__ __forceinline__ void load(const T* x, int64_t e, int64_t n) {
    if constexpr (WIDE) {
      off = 0;
#pragma unroll
      for (int i = 0; i < W; i += 2) ld_global_32(x + e + i * N, q[i], q[i + 1]);
      return;
    }
    off = (int)(e % N);
    const int64_t c = e - off;
    if (c + (W + (off != 0)) * N <= n) {
#pragma unroll
      for (int i = 0; i < W; ++i) q[i] = __ldg(reinterpret_cast<const uint4*>(x + c) + i);
      if (off != 0) q[W] = __ldg(reinterpret_cast<const uint4*>(x + c) + W);
    } else {
      alignas(16) T t[16];
#pragma unroll
      for (int k = 0; k < 16; ++k) t[k] = e + k < n ? x[e + k] : from_f32<T>(0.0f);
#pragma unroll
      for (int i = 0; i < W; ++i) q[i] = reinterpret_cast<const uint4*>(t)[i];
      off = 0;
    }
  }
  __device__ __forceinline__ void get(float (&v)[16]) {
    if (!WIDE && off != 0) {
      uint32_t w[4 * W + 4];
#pragma unroll
      for (int i = 0; i <= W; ++i) {
        w[4 * i] = q[i].x;
        w[4 * i + 1] = q[i].y;
        w[4 * i + 2] = q[i].z;
        w[4 * i + 3] = q[i].w;
      }
      shift_words<4 * W + 4, 4 * W>(w, off * (int)sizeof(T));
#pragma unroll
      for (int i = 0; i < W; ++i) q[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    }
#pragma unroll
    for (int i = 0; i < W; ++i) {
      float f[N];
      unpack<T>(q[i], f);
#pragma unroll
      for (int k = 0; k < N; ++k) v[i * N + k] = f[k];
    }
  }
};

// A thread takes pieces of 16 elements: blockDim.x pieces of a row at a time, blockDim.y rows. Rows are padded to
// whole 128s and columns to whole scale tiles, so that every byte of the scale tiles is written. Pieces of a
// padded row come in multiples of four (NVFP4) or eight (MXFP4) and blockDim.x is a power of two from 8, so the
// pieces of one 32-element block and of one row of a scale tile sit in neighbouring lanes.
template <int FMT, typename T, bool WIDE>
__global__ void __launch_bounds__(MQ_THREADS)
    mx_quantize_kernel(int rows, int64_t row_end, int K, int segs, int64_t col_tiles, int64_t row_bytes,
                       const T* __restrict__ x, const float* __restrict__ gs, uint8_t* __restrict__ codes,
                       uint8_t* __restrict__ sf_out) {
  constexpr int B = MxFormat<FMT>::kBlock, P = B / 16;  // pieces a block
  pdl_wait();
  pdl_trigger();
  const float g = FMT == FP4MOE_W_NVFP4 ? __ldg(gs) : 1.0f;
  const int64_t n = (int64_t)rows * K;
  const int seg = blockIdx.x * blockDim.x + threadIdx.x;
  const int left = K - seg * 16;  // elements of a row from this piece on
  const int64_t step = (int64_t)gridDim.y * blockDim.y;
  int64_t r = (int64_t)blockIdx.y * blockDim.y + threadIdx.y;
  Piece16<T, WIDE> piece;
  auto fetch = [&](int64_t row) {
    if (row < rows && left > 0) piece.load(x, row * K + (int64_t)seg * 16, n);
  };
  fetch(r);
  for (; r < row_end; r += step) {
    const bool any = r < rows && left > 0;
    float v[16];
    // The next row's load goes out as soon as its registers are free: after the unpacking, which shifts and widens,
    // or after a copy where the piece is only eight registers (8192 x 4096 bf16 to NVFP4 16.3 against 18.5 us;
    // unaligned and fp32 pieces are better unpacked first, 4096 x 4095 fp32 14.5 against 18.5 us).
    if constexpr (WIDE && sizeof(T) == 2) {
      Piece16<T, WIDE> cur = piece;
      fetch(r + step);
      if (any) cur.get(v);
    } else {
      if (any) piece.get(v);
      fetch(r + step);
    }
    if (left < 16 || !any) {
#pragma unroll
      for (int k = 0; k < 16; ++k) v[k] = any && k < left ? v[k] : 0.0f;
    }
    uint32_t lo, hi;
    uint32_t sf = quantize16<FMT>(v, g, lo, hi);
    if (r < rows && (int64_t)seg * 8 < row_bytes)
      *reinterpret_cast<uint2*>(codes + (size_t)r * row_bytes + (size_t)seg * 8) = make_uint2(lo, hi);
    // the four scale bytes of a tile row in one store
    if (!any || (seg % P) != 0) sf = 0;
    sf <<= 8 * ((seg / P) % 4);
#pragma unroll
    for (int o = P; o < 4 * P; o <<= 1) sf |= __shfl_xor_sync(0xFFFFFFFFu, sf, o);
    if (seg % (4 * P) == 0 && seg < segs)
      *reinterpret_cast<uint32_t*>(sf_out + mx_sf_offset((uint64_t)r, (uint32_t)(seg / P), (uint64_t)col_tiles)) = sf;
  }
}

// Two E2M1 codes of a byte as fp32, the low nibble first.
__device__ __forceinline__ float2 e2m1x2_to_f32(uint32_t byte) {
  uint32_t h;
  asm("{\n\t.reg .b8 b;\n\tcvt.u8.u32 b, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, b;\n\t}" : "=r"(h) : "r"(byte));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// The values of a piece of one block, 32 bytes of T: sixteen codes of a 16-bit type (w0 the first eight) or eight of
// fp32. MXFP4 e2m1 * s, exact; NVFP4 RN(e2m1 * s / g). A block has the magnitudes 2^e and 1.5 * 2^e only, and a
// power of two commutes with the rounding while nothing leaves the normal range, so two divisions serve a piece:
// t1 = RN(s / g), t15 = RN(1.5 s / g). 16-bit types look the eight magnitudes up in registers, four codes at a
// time: __byte_perm takes the low three bits of each nibble as the index of one of eight bytes.
template <int FMT, typename T>
__device__ __forceinline__ void piece_values(uint32_t w0, uint32_t w1, uint32_t byte, float g, uint32_t (&out)[8]) {
  const float s = mx_scale<FMT>(byte);
  float t1 = s, t15 = 1.5f * s;
  bool exact = true;
  if constexpr (FMT == FP4MOE_W_NVFP4) {
    t1 = __fdiv_rn(s, g);
    t15 = __fdiv_rn(1.5f * s, g);
    const float a = fabsf(t1);
    exact = (a >= 0x1p-100f && a <= 0x1p100f) || (s == 0.0f && a == 0.0f);  // a block of zeros is zeros
  }
  if constexpr (sizeof(T) == 2) {
    float mag[8] = {0.0f, 0.5f * t1, t1, t15, 2.0f * t1, 2.0f * t15, 4.0f * t1, 4.0f * t15};
    if (FMT == FP4MOE_W_MXFP4 && byte == 255u) mag[0] = s;  // a NaN block is NaN throughout
    if (!exact) {
#pragma unroll
      for (uint32_t m = 0; m < 8; ++m) mag[m] = __fdiv_rn(e2m1_to_f32(m) * s, g);
    }
    uint32_t p[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = pack2<T>(mag[2 * i], mag[2 * i + 1]);
    const uint32_t lo0 = __byte_perm(p[0], p[1], 0x6420), lo1 = __byte_perm(p[2], p[3], 0x6420);
    const uint32_t hi0 = __byte_perm(p[0], p[1], 0x7531), hi1 = __byte_perm(p[2], p[3], 0x7531);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t c = (i < 2 ? w0 : w1) >> (16 * (i & 1));
      const uint32_t lo = __byte_perm(lo0, lo1, c & 0x7777u), hi = __byte_perm(hi0, hi1, c & 0x7777u);
      out[2 * i] = __byte_perm(lo, hi, 0x5140) ^ (((c & 0x8u) << 12) | ((c & 0x80u) << 24));
      out[2 * i + 1] = __byte_perm(lo, hi, 0x7362) ^ (((c & 0x800u) << 4) | ((c & 0x8000u) << 16));
    }
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 f = e2m1x2_to_f32((w0 >> (8 * k)) & 0xFFu);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float m = h ? f.y : f.x;
        float v;
        if (FMT == FP4MOE_W_MXFP4) {
          v = m * s;
        } else if (exact) {
          const uint32_t b = __float_as_uint(m);  // its power of two, and whether 1.5 multiplies it
          v = __uint_as_float(b & 0xFF800000u) * ((b & 0x00400000u) ? t15 : t1);
        } else {
          v = __fdiv_rn(m * s, g);
        }
        out[2 * k + h] = __float_as_uint(v);
      }
    }
  }
}

// The first `bytes` (even, less than 16) of v to p, which lies as far before a 16-byte boundary.
__device__ __forceinline__ void store_head(uint8_t* p, uint4 v, int bytes) {
  if (bytes & 2) {
    *reinterpret_cast<uint16_t*>(p) = (uint16_t)v.x;
    v = make_uint4(__byte_perm(v.x, v.y, 0x5432), __byte_perm(v.y, v.z, 0x5432), __byte_perm(v.z, v.w, 0x5432), 0);
    p += 2;
  }
  if (bytes & 4) {
    *reinterpret_cast<uint32_t*>(p) = v.x;
    v = make_uint4(v.y, v.z, v.w, 0);
    p += 4;
  }
  if (bytes & 8) *reinterpret_cast<uint2*>(p) = make_uint2(v.x, v.y);
}
// The same for p on a 16-byte boundary.
__device__ __forceinline__ void store_tail(uint8_t* p, uint4 v, int bytes) {
  if (bytes & 8) {
    *reinterpret_cast<uint2*>(p) = make_uint2(v.x, v.y);
    v = make_uint4(v.z, v.w, 0, 0);
    p += 8;
  }
  if (bytes & 4) {
    *reinterpret_cast<uint32_t*>(p) = v.x;
    v.x = v.y;
    p += 4;
  }
  if (bytes & 2) *reinterpret_cast<uint16_t*>(p) = (uint16_t)v.x;
}

// A thread takes 32 bytes of output, E values of one block, in threads and rows as in mx_quantize_kernel, and the
// next row's codes are in flight meanwhile. WIDE: one 32-byte store. SHIFT: rows start at any element of a
// 16-byte vector of the output (off = the row's first element modulo the vector). A lane then takes the last `off`
// values of the lane before and leaves its own last ones to the next, so whole vectors are stored at their
// boundaries. What no whole vector holds, at the ends of a row and of a warp's share of it, goes in smaller stores.
template <int FMT, typename T, bool SHIFT, bool WIDE>
__global__ void __launch_bounds__(MQ_THREADS)
    mx_dequantize_kernel(int rows, int K, int64_t col_tiles, int64_t row_bytes, const uint8_t* __restrict__ codes,
                         const uint8_t* __restrict__ sf, const float* __restrict__ gs, T* __restrict__ out) {
  constexpr int B = MxFormat<FMT>::kBlock, E = 32 / (int)sizeof(T), N = E / 2;
  pdl_wait();
  pdl_trigger();
  const float g = FMT == FP4MOE_W_NVFP4 ? __ldg(gs) : 1.0f;
  const int seg = blockIdx.x * blockDim.x + threadIdx.x;
  const int e0 = E * seg;  // first element
  const int64_t step = (int64_t)gridDim.y * blockDim.y;
  uint2 nc = make_uint2(0, 0);
  uint32_t nb = 0;
  auto fetch = [&](int64_t r) {
    if (r < rows && e0 < K) {
      const uint8_t* p = codes + (size_t)r * row_bytes + E / 2 * (size_t)seg;
      if constexpr (E == 16)
        nc = __ldg(reinterpret_cast<const uint2*>(p));
      else
        nc.x = __ldg(reinterpret_cast<const uint32_t*>(p));
      nb = __ldg(sf + mx_sf_offset((uint64_t)r, (uint32_t)(e0 / B), (uint64_t)col_tiles));
    }
  };
  int64_t rb = (int64_t)blockIdx.y * blockDim.y;  // the lanes of a warp loop alike, whatever their rows
  fetch(rb + threadIdx.y);
  for (; rb < rows; rb += step) {
    const int64_t r = rb + threadIdx.y;
    uint32_t v[8];
    const uint2 c = nc;
    const uint32_t byte = nb;
    fetch(r + step);
    piece_values<FMT, T>(c.x, c.y, byte, g, v);
    const uint4 a = make_uint4(v[0], v[1], v[2], v[3]), b = make_uint4(v[4], v[5], v[6], v[7]);
    T* row = out + (size_t)r * K;
    if constexpr (!SHIFT) {
      if (r < rows && e0 < K) {
        if constexpr (WIDE) {
          st_global_32(row + e0, a, b);
        } else {  // K is a multiple of N
          *reinterpret_cast<uint4*>(row + e0) = a;
          if (e0 + N < K) *reinterpret_cast<uint4*>(row + e0 + N) = b;
        }
      }
    } else {
      const int lane = (int)((threadIdx.y * blockDim.x + threadIdx.x) & 31u);
      const int off = (int)(r * K % N), bytes = off * (int)sizeof(T);
      uint32_t w[12];
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = __shfl_up_sync(0xFFFFFFFFu, v[4 + i], 1);
#pragma unroll
      for (int i = 0; i < 8; ++i) w[4 + i] = v[i];
      if (off > 0) {
        shift_words<12, 8>(w, 16 - bytes);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = w[i + 4];
      }
      if (r < rows && e0 < K) {
        // first: no lane before; e: the piece's first vector, which begins in the lane before where off > 0
        const bool first = seg == 0 || lane == 0;
        const int e = e0 - off;
        if (e0 + E <= K) {
          if (!first || off == 0)
            *reinterpret_cast<uint4*>(row + e) = make_uint4(w[0], w[1], w[2], w[3]);
          else
            store_head(reinterpret_cast<uint8_t*>(row + e0), a, 16 - bytes);
          *reinterpret_cast<uint4*>(row + e + N) = make_uint4(w[4], w[5], w[6], w[7]);
          // the last `off` values, where the next lane has no whole vector for them
          if (off > 0 && (lane == 31 || e0 + E - off + N > K)) {
            uint32_t t[8] = {v[4], v[5], v[6], v[7], 0, 0, 0, 0};
            shift_words<8, 4>(t, 16 - bytes);
            store_tail(reinterpret_cast<uint8_t*>(row + e0 + E - off), make_uint4(t[0], t[1], t[2], t[3]), bytes);
          }
        } else {  // the row's last piece, cut short
          alignas(16) T own[E];
          *reinterpret_cast<uint4*>(own) = a;
          *reinterpret_cast<uint4*>(own + N) = b;
          const bool whole = e + N <= K && (!first || off == 0);
          if (whole) *reinterpret_cast<uint4*>(row + e) = make_uint4(w[0], w[1], w[2], w[3]);
#pragma unroll
          for (int k = 0; k < E; ++k)
            if (e0 + k < K && (!whole || e0 + k >= e + N)) row[e0 + k] = own[k];
        }
      }
    }
  }
}

// Threads and CTAs for `rows` rows of `pieces` pieces: blockDim.x a power of two from 8 that holds a row if 256 do,
// the other threads on further rows.
struct Shape {
  dim3 grid, block;
};
Shape row_shape(int64_t rows, int64_t pieces, int ctas_per_sm) {
  unsigned tx = 8;
  while (tx < MQ_THREADS && tx < pieces) tx *= 2;
  const unsigned ty = MQ_THREADS / tx;
  const int64_t gx = (pieces + tx - 1) / tx, want = (rows + ty - 1) / ty;
  const int64_t fill = std::max<int64_t>(1, (int64_t)sm_count() * ctas_per_sm / gx);
  return {dim3((unsigned)gx, (unsigned)std::min<int64_t>({want, fill, 65535})), dim3(tx, ty)};
}

template <int FMT, typename T>
fp4moe_status quantize_launch(int32_t rows, int32_t K, const void* x, const float* gs, uint8_t* codes, uint8_t* sf,
                              cudaStream_t st) {
  const int64_t ct = mx_col_tiles(FMT, K), segs = ct * 4 * MxFormat<FMT>::kBlock / 16;
  const int64_t row_end = mx_row_tiles(rows) * 128;
  const Shape s = row_shape(row_end, segs, kCtasPerSm);
  const bool wide = K % 16 == 0 && (reinterpret_cast<uintptr_t>(x) & 31u) == 0;
  return launch_pdl(wide ? mx_quantize_kernel<FMT, T, true> : mx_quantize_kernel<FMT, T, false>, s.grid, s.block, 0,
                    st, rows, row_end, K, (int)segs, ct, mx_row_bytes(K), static_cast<const T*>(x), gs, codes,
                    sf) == cudaSuccess
             ? FP4MOE_OK
             : FP4MOE_CUDA_ERROR;
}

template <int FMT, typename T>
fp4moe_status dequantize_launch(int32_t rows, int32_t K, const uint8_t* codes, const uint8_t* sf, const float* gs,
                                void* out, cudaStream_t st) {
  const bool shift = K % (16 / sizeof(T)) != 0;
  const Shape s = row_shape(rows, ((int64_t)K * (int)sizeof(T) + 31) / 32, kCtasPerSmInverse);
  const bool wide = K % 16 == 0 && (reinterpret_cast<uintptr_t>(out) & 31u) == 0;
  return launch_pdl(shift  ? mx_dequantize_kernel<FMT, T, true, false>
                    : wide ? mx_dequantize_kernel<FMT, T, false, true>
                           : mx_dequantize_kernel<FMT, T, false, false>,
                    s.grid, s.block, 0, st, rows, K, mx_col_tiles(FMT, K), mx_row_bytes(K), codes, sf, gs,
                    static_cast<T*>(out)) == cudaSuccess
             ? FP4MOE_OK
             : FP4MOE_CUDA_ERROR;
}

}  // namespace

fp4moe_status mx_quantize_launch(int32_t format, int32_t dtype, int32_t rows, int32_t K, const void* x,
                                 const float* gs, uint8_t* codes, uint8_t* sf, cudaStream_t st) {
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
