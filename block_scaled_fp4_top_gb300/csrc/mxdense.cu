// Dense product of two microscaled 4-bit matrices:  out[M][N] = alpha * A[M][K] . B[N][K]^T.
//
// Both operands are E2M1 codes with one E8M0 scale per 32 elements (MXFP4) or one E4M3 scale per 16 (NVFP4),
// in the layouts that mxquant.cu writes. The tensor cores multiply them with their scales
// (tcgen05.mma kind::mxf4nvf4.block_scale, K = 64 per instruction, scale_vec::2X or ::4X) and add in fp32; the
// epilogue multiplies by alpha and rounds once to the output type. Bytes: (M + N) K (1/2 + 1/32 or 1/16) in,
// M N out; 2 M N K flops.
//
// A CTA owns one 128 x BN output tile at a time (BN weight rows), walking the tiles with a static stride.
//   warps 0-7   epilogue (warp w: TMEM lanes 32 (w % 4) .., columns BN / 2 * (w / 4) ..).
//   warp 8      producer: a ring stage is 256 K elements of A and B by TMA (128-byte swizzle) and their scale
//               tiles, which a second pair of tensor maps views as rows of 512 bytes. Rows and columns past the
//               matrices arrive as zeros.
//   warp 9      MMA issuer, one thread.
//   warps 10-11 scale copiers: tcgen05.cp of the stage's scale tiles into the stage's TMEM slot.
// The accumulator takes BN TMEM columns; the epilogue moves it whole to registers and frees it before it
// computes, so the next tile's MMAs wait only for that move.
//
// A 128 x 4 scale tile spans 64 K elements in NVFP4, one MMA, and 128 in MXFP4, two MMAs: there the instruction
// descriptor's scale-factor ids pick bytes 0-1 or 2-3 of each row's four. The last stage of a K that is no
// multiple of 256 issues only the MMAs that hold elements; TMA may load scale tiles of the next row tile behind
// it, which no MMA reads. Elements past K inside an MMA have zero codes and a zero scale byte.
//
// Every wait is bounded (common.cuh): one that runs out sets FP4MOE_ERR_TIMEOUT in the caller's error word,
// copies and MMAs in flight are drained, and the CTA frees its TMEM and returns.
#include <mutex>

#include "common.cuh"
#include "dense.cuh"
#include "internal.h"

namespace fp4moe {

bool encode_u8_sw128(CUtensorMap* m, const void* base, uint64_t inner_bytes, uint64_t rows, uint32_t box_rows);
bool encode_scale_tiles(CUtensorMap* m, const void* base, uint64_t tiles, uint32_t box_tiles);

namespace {

constexpr int DBM = 128;       // rows of A per tile (MMA M)
constexpr int DK = 256;        // K elements per ring stage: 128 bytes of codes, 4 MMAs of K = 64
constexpr int DEPI = 8;        // epilogue warps
constexpr int DNCOPY = 2;      // scale copier warps
constexpr int DTHREADS = 32 * (DEPI + 2 + DNCOPY);
constexpr int DPRODUCER = DEPI, DMMA = DEPI + 1, DCOPY0 = DEPI + 2;
constexpr uint32_t DTMEM_COLS = 512;

// Sizes of one kernel instance.
template <int FMT, int BN>
struct DenseCfg {
  static constexpr int kSfTiles = FMT == FP4MOE_W_MXFP4 ? 2 : 4;  // scale tiles per 128 rows of a stage
  static constexpr int kHalves = BN / 128;
  static constexpr int kA = DBM * 128, kB = BN * 128;
  static constexpr int kSfa = kSfTiles * 512, kSfb = kHalves * kSfTiles * 512;
  static constexpr int kBytes = kA + kB + kSfa + kSfb;
  static constexpr int kStage = (kBytes + 1023) / 1024 * 1024;
  static constexpr int kStages = BN == 256 ? 4 : 6;
  static constexpr int kBarOff = kStages * kStage;
  static constexpr int kSmem = kBarOff + 256 + 1024;  // barriers + 1024-byte alignment slack
  static constexpr uint32_t kSlotCols = 4 * kSfTiles * (1 + kHalves);  // TMEM columns of one stage's scales
  static constexpr int kCopies = kSfTiles * (1 + kHalves);
  static_assert(BN + kSlotCols * kStages <= DTMEM_COLS, "accumulator and scale slots fit TMEM");
  static_assert(kSmem <= 232448 - 64, "shared memory budget");
  static_assert(8 * (3 * kStages + 4) <= 256, "barriers fit their area");
};

struct DenseMaps {
  CUtensorMap a, b, sfa, sfb;
};

struct DenseParams {
  int M, N, K;
  int KB;            // ring stages per tile
  int mt, nt;        // output tiles along M and N
  int ct;            // scale tiles across K
  const float* alpha;
  void* out;
  int vec;           // rows of out start 16-byte aligned
  uint32_t* err;
};

// D[tmem] (+)= A[smem] * B[smem]^T with block scales in TMEM (K = 64).
template <int FMT>
__device__ __forceinline__ void tc_mma_mx(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t sfa,
                                          uint32_t sfb, uint32_t accumulate) {
  if constexpr (FMT == FP4MOE_W_MXFP4)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(
            d),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
  else
    tc_mma_nvf4(d, adesc, bdesc, idesc, sfa, sfb, accumulate);
}

// Instruction descriptor: idesc_nvf4, with E8M0 scales and the scale-factor ids of the MMA's half for MXFP4.
template <int FMT>
__host__ __device__ constexpr uint32_t idesc_mx(int M, int N, uint32_t sf_id) {
  return idesc_nvf4(M, N) | (FMT == FP4MOE_W_MXFP4 ? (1u << 23) | (sf_id << 4) | (sf_id << 29) : 0u);
}

// Columns [0, n) of v into row pointer p (n <= 32): 16-byte stores where the row allows them.
template <typename T>
__device__ __forceinline__ void store_row(T* p, const float* v, int n, bool vec) {
  constexpr int V = 16 / (int)sizeof(T);
  if (vec) {  // n is a multiple of V, or at least 32
#pragma unroll
    for (int i = 0; i < 32; i += V) {
      if (i < n) {
        alignas(16) T t[V];
#pragma unroll
        for (int j = 0; j < V; ++j) t[j] = from_f32<T>(v[i + j]);
        *reinterpret_cast<uint4*>(p + i) = *reinterpret_cast<const uint4*>(t);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (i < n) p[i] = from_f32<T>(v[i]);
  }
}

template <int FMT, int BN, typename T>
__global__ void __launch_bounds__(DTHREADS, 1)
    mx_dense_kernel(const __grid_constant__ DenseMaps maps, const DenseParams prm) {
  using C = DenseCfg<FMT, BN>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t smem = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t bar_full = smem + C::kBarOff;
  const uint32_t bar_empty = bar_full + 8 * C::kStages;
  const uint32_t bar_sready = bar_empty + 8 * C::kStages;
  const uint32_t bar_tfull = bar_sready + 8 * C::kStages;
  const uint32_t bar_tempty = bar_tfull + 8;
  const uint32_t bar_drain = bar_tempty + 8;
  const uint32_t bar_cdrain = bar_drain + 8;

  if (warp == 0) {
    tmem_alloc(smem_u32(&s_tmem), DTMEM_COLS);
    tmem_relinquish();
  }
  if (threadIdx.x == 32 * DPRODUCER) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(bar_full + 8 * s, 1);
      mbar_init(bar_empty + 8 * s, 1);
      mbar_init(bar_sready + 8 * s, DNCOPY);
    }
    mbar_init(bar_tfull, 1);
    mbar_init(bar_tempty, DEPI);
    mbar_init(bar_drain, 1);
    mbar_init(bar_cdrain, DNCOPY);
    fence_mbar_init();
  }
  pdl_wait();
  pdl_trigger();
  if (threadIdx.x == 0) s_abort = (*(volatile uint32_t*)prm.err & kAbortMask) != 0;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  // an earlier timeout poisons the call: no role takes a tile
  const int tiles = s_abort ? 0 : prm.mt * prm.nt;
  const int KB = prm.KB;

  if (warp == DPRODUCER && lane == 0) {
    const uint64_t pol = policy_evict_normal();
    int it = 0;
    bool ok = true;
    for (int t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
      const int m = t % prm.mt, n = t / prm.mt;
      for (int kb = 0; kb < KB; ++kb, ++it) {
        const int s = it % C::kStages;
        if (!mbar_wait(bar_empty + 8 * s, ((uint32_t)(it / C::kStages) & 1u) ^ 1u, prm.err)) {
          ok = false;
          break;
        }
        const uint32_t st = smem + s * C::kStage, full = bar_full + 8 * s;
        mbar_arrive_expect_tx(full, C::kBytes);
        tma_load_2d(st, &maps.a, full, kb * 128, m * DBM, pol);
        tma_load_2d(st + C::kA, &maps.b, full, kb * 128, n * BN, pol);
        tma_load_2d(st + C::kA + C::kB, &maps.sfa, full, 0, m * prm.ct + kb * C::kSfTiles, pol);
#pragma unroll
        for (int h = 0; h < C::kHalves; ++h)
          tma_load_2d(st + C::kA + C::kB + C::kSfa * (1 + h), &maps.sfb, full, 0,
                      (n * C::kHalves + h) * prm.ct + kb * C::kSfTiles, pol);
      }
    }
    // on every path, let the copies already issued land before the CTA exits
    for (int j = max(0, it - C::kStages); j < it; ++j)
      drain_wait(bar_full + 8 * (j % C::kStages), (uint32_t)(j / C::kStages) & 1u);
  } else if (warp == DMMA && lane == 0) {
    int tl = 0, s = 0;
    uint32_t ph = 0;
    bool ok = true;
    for (int t = blockIdx.x; ok && t < tiles; t += gridDim.x, ++tl) {
      // the epilogue has moved the previous tile's accumulator out of TMEM
      if (!mbar_wait(bar_tempty, ((uint32_t)tl & 1u) ^ 1u, prm.err)) break;
      for (int kb = 0; kb < KB; ++kb) {
        if (!mbar_wait(bar_full + 8 * s, ph, prm.err) || !mbar_wait(bar_sready + 8 * s, ph, prm.err)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t st = smem + (uint32_t)s * C::kStage;
        const uint32_t sfa = tmem + BN + C::kSlotCols * s, sfb = sfa + 4 * C::kSfTiles;
        const int atoms = min(4, (prm.K - kb * DK + 63) / 64);
#pragma unroll
        for (int a = 0; a < 4; ++a) {
          if (a < atoms) {
            constexpr bool mx = FMT == FP4MOE_W_MXFP4;
            const int tile = mx ? a >> 1 : a;
            tc_mma_mx<FMT>(tmem, desc_sw128(st + 32 * a), desc_sw128(st + C::kA + 32 * a),
                           idesc_mx<FMT>(DBM, BN, mx ? 2 * (a & 1) : 0), sfa + 4 * tile, sfb + 4 * C::kHalves * tile,
                           (kb > 0 || a > 0) ? 1u : 0u);
          }
        }
        tc_commit(bar_empty + 8 * s);
        if (++s == C::kStages) {
          s = 0;
          ph ^= 1u;
        }
      }
      if (ok) tc_commit(bar_tfull);
    }
    tc_commit(bar_drain);
    drain_wait(bar_drain, 0);  // no MMA may still write TMEM when it is freed
  } else if (warp >= DCOPY0 && lane == 0) {
    // Copy i: A tile i, then B tile j half h at column 4 (kHalves j + h), so that an N = 256 MMA finds the two
    // 128-row halves side by side. TMEM slot s is free once stage s is full again: the producer refilled it
    // only after the MMAs of the slot's previous use committed bar_empty.
    const int cpy = warp - DCOPY0;
    int s = 0;
    uint32_t ph = 0;
    bool ok = true;
    for (int t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
      for (int kb = 0; kb < KB; ++kb) {
        if (!mbar_wait(bar_full + 8 * s, ph, prm.err)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t sf = smem + (uint32_t)s * C::kStage + C::kA + C::kB;
        const uint32_t slot = tmem + BN + C::kSlotCols * s;
#pragma unroll
        for (int i = cpy; i < C::kCopies; i += DNCOPY) {
          if (i < C::kSfTiles) {
            tc_cp_scales(slot + 4 * i, desc_scales(sf + 512 * i));
          } else {
            const int j = (i - C::kSfTiles) / C::kHalves, h = (i - C::kSfTiles) % C::kHalves;
            tc_cp_scales(slot + 4 * C::kSfTiles + 4 * (C::kHalves * j + h),
                         desc_scales(sf + C::kSfa * (1 + h) + 512 * j));
          }
        }
        tc_commit(bar_sready + 8 * s);
        if (++s == C::kStages) {
          s = 0;
          ph ^= 1u;
        }
      }
    }
    tc_commit(bar_cdrain);
    drain_wait(bar_cdrain, 0);  // no copy may still write TMEM when it is freed
  } else if (warp < DEPI) {
    constexpr int W = BN / 2;  // columns of one warp
    const int quarter = warp & 3, half = warp >> 2;
    const float alpha = prm.alpha != nullptr ? __ldg(prm.alpha) : 1.0f;
    int tl = 0;
    for (int t = blockIdx.x; t < tiles; t += gridDim.x, ++tl) {
      const int m = t % prm.mt, n = t / prm.mt;
      const int r0 = m * DBM + quarter * 32;
      const int r = r0 + lane, c0 = n * BN + W * half;
      // the whole warp takes one decision: tcgen05.ld is warp-collective
      if (!__all_sync(0xFFFFFFFFu, mbar_wait(bar_tfull, (uint32_t)tl & 1u, prm.err) ? 1 : 0)) break;
      tc_fence_after();
      const bool live = r0 < prm.M && c0 < prm.N;
      float v[W];
      if (live) {
        const uint32_t tacc = tmem + (uint32_t)(W * half) + ((uint32_t)(quarter * 32) << 16);
#pragma unroll
        for (int c = 0; c < W / 32; ++c) {
          float q[32];
          tmem_ld32(tacc + c * 32, q);
#pragma unroll
          for (int j = 0; j < 32; ++j) v[c * 32 + j] = q[j];
        }
        tmem_ld_wait();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_tempty);  // this warp's share of the accumulator is out of TMEM
      if (live && r < prm.M) {
#pragma unroll
        for (int j = 0; j < W; ++j) v[j] *= alpha;
        T* row = static_cast<T*>(prm.out) + (size_t)r * prm.N;
#pragma unroll
        for (int c = 0; c < W; c += 32)
          if (c0 + c < prm.N) store_row(row + c0 + c, v + c, prm.N - c0 - c, prm.vec != 0);
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, DTMEM_COLS);
  }
}

template <int FMT, int BN, typename T>
bool dense_configure() {
  static int ok = -1;
  static std::once_flag once;
  std::call_once(once, [] {
    ok = cudaFuncSetAttribute(mx_dense_kernel<FMT, BN, T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              DenseCfg<FMT, BN>::kSmem) == cudaSuccess
             ? 1
             : 0;
  });
  return ok == 1;
}

template <int FMT, int BN, typename T>
fp4moe_status dense_run(DenseParams prm, const uint8_t* a, const uint8_t* a_sf, const uint8_t* b, const uint8_t* b_sf,
                        int nsm, cudaStream_t st) {
  using C = DenseCfg<FMT, BN>;
  prm.nt = (prm.N + BN - 1) / BN;
  DenseMaps maps;
  const uint64_t rb = (uint64_t)mx_row_bytes(prm.K);
  if (!encode_u8_sw128(&maps.a, a, rb, (uint64_t)prm.M, DBM) || !encode_u8_sw128(&maps.b, b, rb, (uint64_t)prm.N, BN) ||
      !encode_scale_tiles(&maps.sfa, a_sf, (uint64_t)mx_row_tiles(prm.M) * prm.ct, C::kSfTiles) ||
      !encode_scale_tiles(&maps.sfb, b_sf, (uint64_t)mx_row_tiles(prm.N) * prm.ct, C::kSfTiles))
    return FP4MOE_CUDA_ERROR;
  if (!dense_configure<FMT, BN, T>()) return FP4MOE_CUDA_ERROR;
  const int tiles = prm.mt * prm.nt;
  const unsigned grid = (unsigned)(tiles < nsm ? tiles : nsm);
  return launch_pdl(mx_dense_kernel<FMT, BN, T>, dim3(grid), dim3(DTHREADS), C::kSmem, st, maps, prm) == cudaSuccess
             ? FP4MOE_OK
             : FP4MOE_CUDA_ERROR;
}

template <int FMT, typename T>
fp4moe_status dense_pick(const DenseParams& prm, const uint8_t* a, const uint8_t* a_sf, const uint8_t* b,
                         const uint8_t* b_sf, cudaStream_t st) {
  const int nsm = sm_count();
  if (nsm <= 0) return FP4MOE_CUDA_ERROR;
  // 128 x 256 tiles once they fill the device; smaller products spread over more CTAs with 128 x 128 tiles.
  if ((int64_t)prm.mt * ((prm.N + 255) / 256) >= nsm) return dense_run<FMT, 256, T>(prm, a, a_sf, b, b_sf, nsm, st);
  return dense_run<FMT, 128, T>(prm, a, a_sf, b, b_sf, nsm, st);
}

template <int FMT>
fp4moe_status dense_typed(int32_t dtype, const DenseParams& prm, const uint8_t* a, const uint8_t* a_sf,
                          const uint8_t* b, const uint8_t* b_sf, cudaStream_t st) {
  switch (dtype) {
    case FP4MOE_BF16:
      return dense_pick<FMT, __nv_bfloat16>(prm, a, a_sf, b, b_sf, st);
    case FP4MOE_FP16:
      return dense_pick<FMT, __half>(prm, a, a_sf, b, b_sf, st);
    default:
      return dense_pick<FMT, float>(prm, a, a_sf, b, b_sf, st);
  }
}

}  // namespace

fp4moe_status mx_dense_launch(int32_t format, int32_t dtype, int32_t M, int32_t N, int32_t K, const uint8_t* a,
                              const uint8_t* a_sf, const uint8_t* b, const uint8_t* b_sf, const float* alpha,
                              void* out, uint32_t* err, cudaStream_t st) {
  DenseParams prm{};
  prm.M = M;
  prm.N = N;
  prm.K = K;
  prm.KB = (K + DK - 1) / DK;
  prm.mt = (M + DBM - 1) / DBM;
  prm.ct = (int)mx_col_tiles(format, K);
  prm.alpha = alpha;
  prm.out = out;
  prm.vec = ((int64_t)N * (dtype == FP4MOE_FP32 ? 4 : 2)) % 16 == 0 ? 1 : 0;
  prm.err = err;
  return format == FP4MOE_W_MXFP4 ? dense_typed<FP4MOE_W_MXFP4>(dtype, prm, a, a_sf, b, b_sf, st)
                                  : dense_typed<FP4MOE_W_NVFP4>(dtype, prm, a, a_sf, b, b_sf, st);
}

}  // namespace fp4moe
