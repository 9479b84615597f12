// Shared parts of the dense 4-bit products (mxdense.cu, mxpair.cu).
#pragma once

#include "common.cuh"
#include "dense.cuh"
#include "perdevice.h"

namespace fp4moe {

bool encode_u8_sw128(CUtensorMap* m, const void* base, uint64_t inner_bytes, uint64_t rows, uint32_t box_rows);

constexpr int DK = 256;  // K elements per ring stage: 128 bytes of codes, 4 MMAs of K = 64

struct DenseMaps {
  CUtensorMap a, b, sfa, sfb;
};

struct DenseParams {
  int M, N, K;
  int KB;      // ring stages per tile
  int mt, nt;  // output tiles along M and N
  int ct;      // scale tiles across K
  const uint8_t *a_sf, *b_sf;  // scale tiles (mxdense.cu)
  const float* alpha;
  void* out;
  int vec;     // log2 of the bytes that rows of out are aligned to: 5, 4, 2 or 1
  uint32_t* err;
};

// 16 bytes to an address of another CTA of the cluster, counted on a barrier there (both from map_cluster).
__device__ __forceinline__ void st_async_16(uint32_t caddr, float a, float b, float c, float d, uint32_t cbar) {
  asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(
                   caddr),
               "r"(__float_as_uint(a)), "r"(__float_as_uint(b)), "r"(__float_as_uint(c)), "r"(__float_as_uint(d)),
               "r"(cbar)
               : "memory");
}

// Arrive on a barrier of any CTA of the cluster (an address from map_cluster), and the same with bytes to come.
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t caddr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(caddr) : "memory");
}
__device__ __forceinline__ void mbar_arrive_expect_tx_cluster(uint32_t caddr, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cluster.b64 _, [%0], %1;" ::"r"(caddr), "r"(bytes) : "memory");
}

__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"((uint64_t)map) : "memory");
}

// One lane of a converged warp. The warps that issue MMAs run their loops in all lanes, with one elected lane around
// the tcgen05 instructions alone: descriptors and addresses then stay in uniform registers, which those
// instructions take. Loops inside a one-lane branch move ten values per MMA between register files, and a MMA of
// 128 cycles was issued every 180.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}
// mbar_wait in all lanes of a converged warp: one answer.
__device__ __forceinline__ bool mbar_wait_warp(uint32_t bar, uint32_t parity, uint32_t* err) {
  return __all_sync(0xFFFFFFFFu, mbar_wait(bar, parity, err) ? 1 : 0) != 0;
}

// Instruction descriptor: idesc_nvf4, with E8M0 scales and the scale-factor ids of the MMA's half for MXFP4.
template <int FMT>
__host__ __device__ constexpr uint32_t idesc_mx(int M, int N, uint32_t sf_id) {
  return idesc_nvf4(M, N) | (FMT == FP4MOE_W_MXFP4 ? (1u << 23) | (sf_id << 4) | (sf_id << 29) : 0u);
}

// Bytes of the staging area of one epilogue warp: 32 rows of 64 bytes.
constexpr int kEpiStage = 32 * 64;

// W columns of a warp's 32 rows (TMEM lanes of its quarter, from column address `tacc`), times alpha, as packed
// words of T. 16-bit types are packed as they arrive: fp32 columns of a whole tile do not fit the registers.
template <typename T, int W>
__device__ __forceinline__ void load_packed(uint32_t tacc, float alpha, uint32_t (&w)[W * sizeof(T) / 4]) {
  constexpr int STEP = W < 64 ? W : 64;
#pragma unroll
  for (int c = 0; c < W; c += STEP) {
    float q[STEP / 32][32];
#pragma unroll
    for (int i = 0; i < STEP / 32; ++i) tmem_ld32(tacc + c + 32 * i, q[i]);
    tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < STEP / 32; ++i) {
      if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int j = 0; j < 32; ++j) w[c + 32 * i + j] = __float_as_uint(q[i][j] * alpha);
      } else {
#pragma unroll
        for (int j = 0; j < 16; ++j)
          w[(c + 32 * i) / 2 + j] = pack2<T>(q[i][2 * j] * alpha, q[i][2 * j + 1] * alpha);
      }
    }
  }
}

// A warp's 32 rows x 64 bytes of output (w: the lane's row; rows r0 + lane, columns c0 ..). vec: log2 of the bytes
// that rows of the output are aligned to (1, 2, 4 or 5). Rows on 32-byte boundaries are stored from registers, whole
// sectors. Others go by way of shared memory, so that a store instruction covers 64-byte pieces of rows instead of
// an element or 16 bytes of 32 rows: 8192 x 4097 x 4096 in tiles of 128 x 128 took 80 us instead of 304, and takes 55
// in those of 256 x 256, where 4096 columns take 45. The 16-byte chunk j of row i lies at i * 64 + (j ^ (i / 2 % 4)) *
// 16: both sides are free of bank conflicts.
template <typename T>
__device__ __forceinline__ void store_chunk(uint8_t* stage, const uint32_t* w, T* out, int M, int N, int r0, int c0,
                                            int lane, int vec) {
  constexpr int V = 16 / (int)sizeof(T), COLS = 64 / (int)sizeof(T);
  if (vec == 5) {
    if (r0 + lane < M) {
      T* p = out + (size_t)(r0 + lane) * N + c0;
#pragma unroll
      for (int j = 0; j < 16; j += 8)
        if (c0 + j * 4 / (int)sizeof(T) < N)
          st_global_32(p + j * 4 / (int)sizeof(T), make_uint4(w[j], w[j + 1], w[j + 2], w[j + 3]),
                       make_uint4(w[j + 4], w[j + 5], w[j + 6], w[j + 7]));
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j)
    *reinterpret_cast<uint4*>(stage + lane * 64 + ((j ^ (lane >> 1 & 3)) << 4)) =
        make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
  __syncwarp();
  const int rows = min(32, M - r0), cols = min(COLS, N - c0);
  T* base = out + (size_t)r0 * N + c0;
  if (vec == 4) {  // four lanes a row; cols is a multiple of V
    const int j = lane & 3;
    if (j * V < cols) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = 8 * i + (lane >> 2);
        if (r < rows)
          *reinterpret_cast<uint4*>(base + (size_t)r * N + j * V) =
              *reinterpret_cast<const uint4*>(stage + r * 64 + ((j ^ (r >> 1 & 3)) << 4));
      }
    }
  } else if (vec == 2) {  // one word a lane, two rows at a time; cols is a multiple of 4 / sizeof(T)
    constexpr int P = 4 / (int)sizeof(T);
    const int c = lane & 15;
    if (c * P < cols) {
#pragma unroll 8
      for (int r = lane >> 4; r < rows; r += 2)
        *reinterpret_cast<uint32_t*>(base + (size_t)r * N + c * P) =
            *reinterpret_cast<const uint32_t*>(stage + r * 64 + (((c >> 2) ^ (r >> 1 & 3)) << 4) + (c & 3) * 4);
    }
  } else if (lane < cols) {  // 16-bit types: one element a lane, a row at a time
#pragma unroll 8
    for (int r = 0; r < rows; ++r)
      reinterpret_cast<uint16_t*>(base)[(size_t)r * N + lane] =
          *reinterpret_cast<const uint16_t*>(stage + r * 64 + (((lane >> 3) ^ (r >> 1 & 3)) << 4) + (lane & 7) * 2);
  }
  __syncwarp();
}

// mxpair.cu: 256 x 256 tiles on CTA pairs. prm.mt and prm.nt are set there.
fp4moe_status mx_pair_launch(int32_t format, int32_t dtype, const DenseParams& prm, const uint8_t* a,
                             const uint8_t* a_sf, const uint8_t* b, const uint8_t* b_sf, cudaStream_t st);

}  // namespace fp4moe
