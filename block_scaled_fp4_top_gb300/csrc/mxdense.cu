// Dense product of two microscaled 4-bit matrices:  out[M][N] = alpha * A[M][K] . B[N][K]^T.
//
// Both operands are E2M1 codes with one E8M0 scale per 32 elements (MXFP4) or one E4M3 scale per 16 (NVFP4),
// in the layouts that mxquant.cu writes. The tensor cores multiply them with their scales
// (tcgen05.mma kind::mxf4nvf4.block_scale, K = 64 per instruction, scale_vec::2X or ::4X) and add in fp32; the
// epilogue multiplies by alpha and rounds once to the output type. Bytes: (M + N) K (1/2 + 1/32 or 1/16) in,
// M N out; 2 M N K flops.
//
// This file holds the kernel for the small sizes, tiles of 128 x 64 or 128 x 128 on single CTAs, and the choice between
// them and the large tiles of mxpair.cu.
//   warps 0-7   epilogue (warp w: TMEM lanes 32 (w % 4) .., half of the columns).
//   warps 8, 9  producers, of A and of B: a ring stage is 256 K elements of both by TMA (128-byte swizzle; of A only
//               the leading 16, 32, 64 or 128 rows that hold M; rows and columns past the matrices arrive as
//               zeros) and their scale tiles by bulk copies.
//   warp 10     per stage, tcgen05.cp of the scale tiles into the stage's TMEM slot, then the MMAs.
// A stage takes about 260 ns whatever its width (four MMAs of at least 65 cycles, the scale copies and the barriers
// around them), so a product with fewer tiles than SMs splits K over a cluster of S CTAs. The CTAs of ranks 1 .. send
// their fp32 partial tiles into buffers of rank 0's shared memory (st.async, counted in bytes on a barrier there),
// and rank 0 adds them to its own in rank order: deterministic, and one trip between SMs instead of a barrier of the
// cluster, a trip there and back and another barrier (1.8 us for one row).
// With more tiles than SMs the grid walks them with a static stride, and the epilogue moves the accumulator to
// registers before the next tile's MMAs need it.
//
// A 128 x 4 scale tile spans 64 K elements in NVFP4, one MMA, and 128 in MXFP4, two MMAs: there the instruction
// descriptor's scale-factor ids pick bytes 0-1 or 2-3 of each row's four. The last stage of a K that is no
// multiple of 256 issues only the MMAs that hold elements, and loads the scale tiles that exist. Elements past K
// inside an MMA have zero codes and a zero scale byte. Rows of A that were
// not loaded, and their scales, are whatever shared memory held: rows of an MMA are independent, and these are
// dropped.
//
// Every wait is bounded (common.cuh): one that runs out sets FP4MOE_ERR_TIMEOUT in the caller's error word,
// copies and MMAs in flight are drained, and the CTA frees its TMEM and returns.
#include <algorithm>
#include <climits>

#include "internal.h"
#include "mxdense.cuh"

namespace fp4moe {
namespace {

constexpr int DBM = 128;          // rows of A per tile (MMA M); BN rows of B (MMA N)
constexpr int DEPI = 8;           // epilogue warps
constexpr int DPRODUCER = DEPI, DMMA = DEPI + 2;  // two producer warps
constexpr int DTHREADS = 32 * (DEPI + 3);
constexpr int kSmemMax = 232448;  // shared memory of a CTA

struct TileMaps {
  CUtensorMap a, b;
};

template <int FMT, int BN>
struct DenseCfg {
  static constexpr int kSfTiles = FMT == FP4MOE_W_MXFP4 ? 2 : 4;  // scale tiles per 128 rows of a stage
  static_assert(BN % 64 == 0, "scale addresses are even");
  static constexpr int kB = BN * 128;
  static constexpr int kSf = kSfTiles * 512;
  // Bytes of a stage: A's rows that are loaded (16, 32, 64 or 128 of 128 bytes), B, the scales. The MMA reads 128
  // rows of A all the same; what follows the loaded ones gives rows that are dropped.
  __host__ __device__ static constexpr int stage(int a_rows) { return a_rows * 128 + kB + 2 * kSf; }
  static constexpr int kMaxStages = 8;
  static constexpr uint32_t kSlotCols = 4 * kSfTiles * 2;  // TMEM columns of one stage's scales
  // Shared memory: a ring of n stages, the rows of A that the last stage's MMAs read past it, S - 1 partial tiles of
  // `a_rows` rows, staging, barriers.
  __host__ __device__ static constexpr int tail(int a_rows) {
    const int past = (DBM - a_rows) * 128 - kB - 2 * kSf;
    return past > 0 ? past : 0;
  }
  __host__ __device__ static constexpr int parts(int S, int a_rows) { return (S - 1) * a_rows * BN * 4; }
  static constexpr int smem(int n, int a_rows, int S) {
    return n * stage(a_rows) + tail(a_rows) + parts(S, a_rows) + DEPI * kEpiStage + 256;
  }
  static constexpr uint32_t tmem(int n) {
    const uint32_t cols = BN + kSlotCols * (uint32_t)n;
    return cols <= 128 ? 128u : cols <= 256 ? 256u : 512u;
  }
  // stages that fit, 0 if none does
  static int fit(int a_rows, int S) {
    int n = kMaxStages;
    while (n > 0 && (smem(n, a_rows, S) > kSmemMax || BN + kSlotCols * (uint32_t)n > 512u)) --n;
    return n;
  }
  static_assert(stage(16) % 1024 == 0, "stage must keep 1024-byte alignment");
  static_assert(8 * (2 * kMaxStages + 4) <= 240, "barriers fit their area");
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

// Where a partial tile holds the 16-byte chunk j of its row i: free of bank conflicts.
template <int BN>
__device__ __forceinline__ uint32_t part_chunk(int i, int j) {
  return (uint32_t)(i * BN * 4 + (j ^ (i & 7)) * 16);
}

// Grid (tiles or persistent CTAs, 1, S), cluster (1, 1, S). stages: ring depth; tmem_cols: a power of two that holds
// the accumulator and the stages' scales.
template <int FMT, int BN, typename T>
__global__ void __launch_bounds__(DTHREADS, 1)
    mx_dense_kernel(const __grid_constant__ TileMaps maps, const DenseParams prm, int stages, int a_rows,
                    uint32_t tmem_cols) {
  using C = DenseCfg<FMT, BN>;
  constexpr int W = BN / 2;  // columns of one epilogue warp
  extern __shared__ __align__(1024) uint8_t smem_raw[];  // all of the CTA's shared memory: no static part shifts it
  const int warp = __shfl_sync(0xFFFFFFFFu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const uint32_t smem = smem_u32(smem_raw);
  const int a_bytes = a_rows * 128, stage_bytes = a_bytes + C::kB + 2 * C::kSf;
  const int S = gridDim.z, z = blockIdx.z;
  const int ring = stages * stage_bytes + C::tail(a_rows), parts = C::parts(S, a_rows);
  uint8_t* const epi_stage = smem_raw + ring + parts;
  const int bar_off = ring + parts + DEPI * kEpiStage;
  const uint32_t bar_full = smem + bar_off;
  const uint32_t bar_empty = bar_full + 8 * C::kMaxStages;
  const uint32_t bar_tfull = bar_empty + 8 * C::kMaxStages;
  const uint32_t bar_tempty = bar_tfull + 8;
  const uint32_t bar_drain = bar_tempty + 8;
  const uint32_t bar_parts = bar_drain + 8;  // rank 0: every epilogue warp of the others has sent its part
  uint32_t& s_tmem = *reinterpret_cast<uint32_t*>(smem_raw + bar_off + 240);
  uint32_t& s_abort = *reinterpret_cast<uint32_t*>(smem_raw + bar_off + 244);
  uint32_t& s_gave_up = *reinterpret_cast<uint32_t*>(smem_raw + bar_off + 248);  // a bit for each epilogue warp

  if (warp == 0) {
    tmem_alloc(smem_u32(&s_tmem), tmem_cols);
    tmem_relinquish();
  }
  if (threadIdx.x == 32 * DPRODUCER) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(bar_full + 8 * s, 2);  // the producers
      mbar_init(bar_empty + 8 * s, 1);
    }
    mbar_init(bar_tfull, 1);
    mbar_init(bar_tempty, DEPI);
    mbar_init(bar_drain, 1);
    mbar_init(bar_parts, S > 1 ? (uint32_t)((S - 1) * DEPI) : 1u);
    fence_mbar_init();
    prefetch_map(&maps.a);
    prefetch_map(&maps.b);
  }
  __syncwarp();
  if (S > 1) cluster_sync();  // rank 0's barrier is ready (before the wait for the previous kernel, which hides it)
  pdl_wait();
  pdl_trigger();
  if (threadIdx.x == 0) {
    s_abort = (*(volatile uint32_t*)prm.err & kAbortMask) != 0 ? 1u : 0u;
    if ((smem & 1023u) != 0) {  // the swizzle needs it, and the compiler grants it
      raise_error(prm.err, FP4MOE_ERR_CAPACITY);
      s_abort = 1u;
    }
    s_gave_up = s_abort ? ~0u : 0u;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, s_tmem, 0);
  // an earlier timeout poisons the call: no role takes a tile
  const int tiles = s_abort ? 0 : prm.mt * prm.nt;
  const int kb0 = prm.KB * z / S, kb1 = prm.KB * (z + 1) / S;  // this slice's stages, one at least

  if ((warp == DPRODUCER || warp == DPRODUCER + 1) && lane == 0) {
    const bool is_b = warp != DPRODUCER;
    const uint64_t pol = policy_evict_normal();
    const uint32_t code_bytes = is_b ? (uint32_t)C::kB : (uint32_t)a_bytes;
    const uint32_t dst = is_b ? (uint32_t)a_bytes : 0u, sf_dst = (uint32_t)(a_bytes + C::kB) + (is_b ? C::kSf : 0u);
    const CUtensorMap* map = is_b ? &maps.b : &maps.a;
    int it = 0, s = 0;
    uint32_t ph = 1;
    bool ok = true;
    for (int t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
      const int row = is_b ? t / prm.mt * BN : t % prm.mt * DBM;
      const uint8_t* sf = (is_b ? prm.b_sf : prm.a_sf) + 512 * (size_t)(row / 128) * prm.ct;
      for (int kb = kb0; kb < kb1; ++kb, ++it) {
        if (!mbar_wait(bar_empty + 8 * s, ph, prm.err)) {
          ok = false;
          break;
        }
        const uint32_t st = smem + s * stage_bytes, full = bar_full + 8 * s;
        const uint32_t sf_bytes = 512u * (uint32_t)min(C::kSfTiles, prm.ct - kb * C::kSfTiles);
        mbar_arrive_expect_tx(full, code_bytes + sf_bytes);
        tma_load_2d(st + dst, map, full, kb * 128, row, pol);
        bulk_load(st + sf_dst, sf + 512 * (size_t)(kb * C::kSfTiles), sf_bytes, full, pol);
        if (++s == stages) {
          s = 0;
          ph ^= 1u;
        }
      }
    }
    // on every path, let the copies already issued land before the CTA exits
    for (int j = max(0, it - stages); j < it; ++j)
      drain_wait(bar_full + 8 * (j % stages), (uint32_t)(j / stages) & 1u);
  } else if (warp == DMMA) {
    const bool leader = elect_one();
    int tl = 0, s = 0;
    uint32_t ph = 0;
    bool ok = true;
    // A scale tile has one TMEM column for 32 rows, and a scale address is even (an odd one raises "misaligned
    // address"), so an output tile begins at row 0 or 64 of a scale tile and none is narrower than 64.
    uint32_t sfb_col = 0;
    auto mma = [&](uint64_t adesc, uint64_t bdesc, uint32_t slot, int a, uint32_t acc) {
      constexpr bool mx = FMT == FP4MOE_W_MXFP4;
      const int tile = mx ? a >> 1 : a;
      tc_mma_mx<FMT>(tmem, adesc + 2 * a, bdesc + 2 * a,
                     idesc_mx<FMT>(DBM, BN, mx ? 2 * (a & 1) : 0), slot + 4 * tile,
                     slot + 4 * C::kSfTiles + 4 * tile + sfb_col, acc);
    };
    for (int t = blockIdx.x; ok && t < tiles; t += gridDim.x, ++tl) {
      // the epilogue has moved the previous tile's accumulator out of TMEM
      if (!mbar_wait_warp(bar_tempty, ((uint32_t)tl & 1u) ^ 1u, prm.err)) break;
      if constexpr (BN < 128) sfb_col = (uint32_t)(t / prm.mt % (128 / BN) * (BN / 32));
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!mbar_wait_warp(bar_full + 8 * s, ph, prm.err)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t st = smem + (uint32_t)(s * stage_bytes), slot = tmem + BN + C::kSlotCols * s;
        const int atoms = (prm.K - kb * DK + 63) / 64;  // of this stage and those behind it
        if (leader) {
          // Copies and MMAs of one thread execute in order, and slot s is free: its last MMAs committed bar_empty.
          // Descriptors hold addresses in units of 16 bytes; within a stage they are added to.
          const uint64_t ad = desc_sw128(st), bd = desc_sw128(st + a_bytes), sd = desc_scales(st + a_bytes + C::kB);
#pragma unroll
          for (int i = 0; i < 2 * C::kSfTiles; ++i) tc_cp_scales(slot + 4 * i, sd + 32 * i);
          if (atoms >= 4) {
#pragma unroll
            for (int a = 0; a < 4; ++a) mma(ad, bd, slot, a, (kb > kb0 || a > 0) ? 1u : 0u);
          } else {
#pragma unroll
            for (int a = 0; a < 3; ++a)
              if (a < atoms) mma(ad, bd, slot, a, (kb > kb0 || a > 0) ? 1u : 0u);
          }
          tc_commit(bar_empty + 8 * s);
        }
        __syncwarp();
        if (++s == stages) {
          s = 0;
          ph ^= 1u;
        }
      }
      if (ok && leader) tc_commit(bar_tfull);
    }
    if (leader) {
      tc_commit(bar_drain);
      drain_wait(bar_drain, 0);  // no MMA may still write TMEM when it is freed
    }
  } else if (warp < DEPI) {
    const int quarter = warp & 3, half = warp >> 2;
    const uint32_t tacc = tmem + (uint32_t)(W * half) + ((uint32_t)(quarter * 32) << 16);
    const float alpha = prm.alpha != nullptr ? __ldg(prm.alpha) : 1.0f;
    int tl = 0;
    for (int t = blockIdx.x; t < tiles; t += gridDim.x, ++tl) {
      const int m = t % prm.mt, n = t / prm.mt;
      const int r0 = m * DBM + quarter * 32, c0 = n * BN + W * half;
      // the whole warp takes one decision: tcgen05.ld is warp-collective
      if (!mbar_wait_warp(bar_tfull, (uint32_t)tl & 1u, prm.err)) {
        if (lane == 0) atomicOr(&s_gave_up, 1u << warp);
        break;
      }
      tc_fence_after();
      const bool live = r0 < prm.M && c0 < prm.N;
      if (S > 1) {  // one tile a cluster
        const int row = quarter * 32 + lane;  // of the tile
        if (z > 0) {
          const uint32_t dst = map_cluster(smem + ring + (z - 1) * a_rows * BN * 4, 0), bar = map_cluster(bar_parts, 0);
          if (lane == 0) mbar_arrive_expect_tx_cluster(bar, live ? min(prm.M - r0, 32) * W * 4 : 0);
          if (live) {
#pragma unroll
            for (int c = 0; c < W; c += 32) {
              float q[32];
              tmem_ld32(tacc + c, q);
              tmem_ld_wait();
              if (r0 + lane < prm.M) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                  st_async_16(dst + part_chunk<BN>(row, (W * half + c) / 4 + j), q[4 * j], q[4 * j + 1], q[4 * j + 2],
                              q[4 * j + 3], bar);
              }
            }
          }
          continue;
        }
        float v[W];
        if (live) {
#pragma unroll
          for (int c = 0; c < W; c += 32) {
            float q[32];
            tmem_ld32(tacc + c, q);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 32; ++j) v[c + j] = q[j];
          }
        }
        if (!mbar_wait_warp(bar_parts, 0, prm.err)) {
          if (lane == 0) atomicOr(&s_gave_up, 1u << warp);
          break;
        }
        if (!live) continue;
        if (row < a_rows) {  // (the rows past M in it hold nothing that is stored)
          for (int p = 0; p < S - 1; ++p) {
            const uint8_t* src = smem_raw + ring + p * a_rows * BN * 4;
#pragma unroll
            for (int j = 0; j < W / 4; ++j) {
              const float4 q = *reinterpret_cast<const float4*>(src + part_chunk<BN>(row, W * half / 4 + j));
              v[4 * j] += q.x;
              v[4 * j + 1] += q.y;
              v[4 * j + 2] += q.z;
              v[4 * j + 3] += q.w;
            }
          }
        }
        constexpr int COLS = 64 / (int)sizeof(T);
#pragma unroll
        for (int c = 0; c < W; c += COLS) {
          uint32_t w[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            if constexpr (sizeof(T) == 4)
              w[j] = __float_as_uint(v[c + j] * alpha);
            else
              w[j] = pack2<T>(v[c + 2 * j] * alpha, v[c + 2 * j + 1] * alpha);
          }
          if (c0 + c < prm.N)
            store_chunk(epi_stage + warp * kEpiStage, w, static_cast<T*>(prm.out), prm.M, prm.N, r0, c0 + c, lane,
                        prm.vec);
        }
        continue;
      }
      uint32_t w[W * sizeof(T) / 4];
      if (live) load_packed<T, W>(tacc, alpha, w);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_tempty);  // this warp's share of the accumulator is out of TMEM
      if (live) {
        constexpr int COLS = 64 / (int)sizeof(T);
#pragma unroll
        for (int c = 0; c < W; c += COLS)
          if (c0 + c < prm.N)
            store_chunk(epi_stage + warp * kEpiStage, w + c * (int)sizeof(T) / 4, static_cast<T*>(prm.out), prm.M,
                        prm.N, r0, c0 + c, lane, prm.vec);
      }
    }
  }

  if (S > 1) {
    __syncwarp();  // the single-thread roles reconverge: cluster barriers are warp-aligned instructions
    cluster_sync();
    // Rank 0 stays until all that was sent to it has landed. The cluster's barrier does not order st.async, so that is
    // bar_parts' phase. Where no warp of rank 0 gave up, its epilogue has waited for it. Else the warps of the other
    // ranks that have not sent their part make up for their arrivals here, so that it completes. (A form of this that
    // sent zeros instead, or in a function of its own, cost calls that end well 0.2 to 0.4 us.)
    if (s_gave_up != 0) {
      if (z > 0) {
        if (lane == 0 && warp < DEPI && (s_gave_up >> warp & 1u) != 0) mbar_arrive_cluster(map_cluster(bar_parts, 0));
      } else if (threadIdx.x == 0) {
        drain_wait(bar_parts, 0);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, tmem_cols);
  }
}

// Rows of A that a tile loads.
int rows_loaded(int M) { return M > 64 ? 128 : M > 32 ? 64 : M > 16 ? 32 : 16; }

// Launch attributes of a split over S CTAs; PDL as in launch_pdl.
cudaLaunchConfig_t dense_config(unsigned grid, int S, size_t smem, cudaStream_t st, cudaLaunchAttribute (&attr)[2]) {
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3(grid, 1, (unsigned)S);
  lc.blockDim = dim3(DTHREADS);
  lc.dynamicSmemBytes = smem;
  lc.stream = st;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 1;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = (unsigned)S;
  lc.attrs = attr;
  lc.numAttrs = S > 1 ? 2 : 1;
  return lc;
}

// The kernel may take all of a CTA's shared memory (an attribute of each device).
template <int FMT, int BN, typename T>
bool dense_configure() {
  static PerDevice done;
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return false;
  return done.get(dev, [] {
    return cudaFuncSetAttribute(mx_dense_kernel<FMT, BN, T>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax) ==
                   cudaSuccess
               ? 1
               : 0;
  }) > 0;
}

// Which kernel, and how. Fitted times of the variants in ns, from back-to-back calls at 55 sizes from 1 x 4096 x 256 to
// 8192 x 8192 x 8192: the one picked is within 7 % of the fastest at all of them (bn64 / bn128 / pair, us: 64 x 8192 x
// 4096 MXFP4 6.8 7.0 9.0, 512 x 4096 x 4096 11.0 7.8 9.3, 768 x 4096 x 4096 15.2 12.0 10.1, 8192 x 4096 x 2048 65 42
// 28.9, 1500 x 3000 x 2000 19 14 10.5; split in two or four 1 x 4096 x 4096 takes 6.0 and 5.6 instead of 6.5, 64 x 4096 x
// 4096 6.4 and 9.9 instead of 6.5, 128 x 2048 x 8192 8.8 and 10.4 instead of 10.1, 128 x 1024 x 14336 11.5 and 10.0
// instead of 15.6). KB: 256-element stages of K.
//   128 x 64, 128 x 128    a launch, 700 a tile and 270 .. 300 a stage
//   split over S CTAs      KB / S stages; joining: 1100 (1600 for tiles of more than 64 rows), and a fifth of a ns for
//                          each fp32 value that is sent
//   256 x 256 on a pair    1050 a tile and 306 a stage, two SMs a tile
MxPlan pick_plan(int M, int N, int KB, int nsm) {
  auto up = [](int64_t a, int64_t b) { return (a + b - 1) / b; };
  MxPlan best{false, 128, 1};
  int64_t best_ns = INT64_MAX;
  auto offer = [&](MxPlan p, int64_t ns) {
    if (ns < best_ns) {
      best_ns = ns;
      best = p;
    }
  };
  for (int bn : {64, 128}) {
    const int64_t tiles = up(M, DBM) * up(N, bn), stage = bn == 128 && M > 64 ? 300 : 270;
    const int64_t launch = bn == 64 ? 1700 : 1800;
    offer({false, bn, 1}, launch + up(tiles, nsm) * (KB * stage + 700));
    if (M > 64 && bn == 128) continue;  // such partial tiles cost more to join than the split saves
    const int64_t rows = std::min(M, DBM), join = M > 64 ? 1600 : 1100;
    for (int S : {2, 4})  // a cluster of four leaves an eighteenth of the SMs without one
      if (S <= KB && tiles * S <= (S == 2 ? nsm : nsm - nsm / 18))
        offer({false, bn, S}, launch + 700 + up(KB, S) * stage + join + (S - 1) * rows * bn / 5);
  }
  offer({true, 256, 1}, 3600 + up(up(M, 256) * up(N, 256), std::max(1, nsm / 2)) * ((int64_t)KB * 306 + 1050));
  return best;
}

template <int FMT, int BN, typename T>
fp4moe_status dense_run(DenseParams prm, int S, const uint8_t* a, const uint8_t* a_sf, const uint8_t* b,
                        const uint8_t* b_sf, int nsm, cudaStream_t st) {
  using C = DenseCfg<FMT, BN>;
  prm.mt = (prm.M + DBM - 1) / DBM;
  prm.nt = (prm.N + BN - 1) / BN;
  const int a_rows = rows_loaded(prm.M);
  const int tiles = prm.mt * prm.nt, ctas = S > 1 ? tiles : std::min(tiles, nsm);
  // as many ring stages as fit, but no more than a CTA's tiles have: the producers run on into the next tile while the
  // epilogue empties the accumulator (1300 x 4100 x 160 MXFP4, one stage a tile: 9.2 with a ring of one, 8.9 us)
  const int64_t work = (int64_t)((prm.KB + S - 1) / S) * ((tiles + ctas - 1) / ctas);
  const int stages = (int)std::min<int64_t>(C::fit(a_rows, S), work);
  if (stages <= 0) return FP4MOE_UNSUPPORTED;  // (not reached: a split in four, the most, leaves room for four stages)
  prm.a_sf = a_sf;
  prm.b_sf = b_sf;
  TileMaps maps;
  const uint64_t rb = (uint64_t)mx_row_bytes(prm.K);
  if (!encode_u8_sw128(&maps.a, a, rb, (uint64_t)prm.M, (uint32_t)a_rows) ||
      !encode_u8_sw128(&maps.b, b, rb, (uint64_t)prm.N, BN))
    return FP4MOE_CUDA_ERROR;
  if (!dense_configure<FMT, BN, T>()) return FP4MOE_CUDA_ERROR;
  cudaLaunchAttribute attr[2];
  const cudaLaunchConfig_t lc = dense_config((unsigned)ctas, S, C::smem(stages, a_rows, S), st, attr);
  return cudaLaunchKernelEx(&lc, mx_dense_kernel<FMT, BN, T>, maps, prm, stages, a_rows, C::tmem(stages)) ==
                 cudaSuccess
             ? FP4MOE_OK
             : FP4MOE_CUDA_ERROR;
}

template <int FMT, int BN>
fp4moe_status dense_typed(int32_t dtype, const DenseParams& prm, int S, const uint8_t* a, const uint8_t* a_sf,
                          const uint8_t* b, const uint8_t* b_sf, int nsm, cudaStream_t st) {
  switch (dtype) {
    case FP4MOE_BF16:
      return dense_run<FMT, BN, __nv_bfloat16>(prm, S, a, a_sf, b, b_sf, nsm, st);
    case FP4MOE_FP16:
      return dense_run<FMT, BN, __half>(prm, S, a, a_sf, b, b_sf, nsm, st);
    default:
      return dense_run<FMT, BN, float>(prm, S, a, a_sf, b, b_sf, nsm, st);
  }
}

template <int FMT>
fp4moe_status dense_width(int bn, int32_t dtype, const DenseParams& prm, int S, const uint8_t* a, const uint8_t* a_sf,
                          const uint8_t* b, const uint8_t* b_sf, int nsm, cudaStream_t st) {
  return bn == 64 ? dense_typed<FMT, 64>(dtype, prm, S, a, a_sf, b, b_sf, nsm, st)
                  : dense_typed<FMT, 128>(dtype, prm, S, a, a_sf, b, b_sf, nsm, st);
}

}  // namespace

MxPlan mx_plan(int M, int N, int K, int sms) { return pick_plan(M, N, (int)(((int64_t)K + DK - 1) / DK), sms); }

fp4moe_status mx_dense_launch(int32_t format, int32_t dtype, int32_t M, int32_t N, int32_t K, const uint8_t* a,
                              const uint8_t* a_sf, const uint8_t* b, const uint8_t* b_sf, const float* alpha,
                              void* out, uint32_t* err, cudaStream_t st) {
  DenseParams prm{};
  prm.M = M;
  prm.N = N;
  prm.K = K;
  prm.KB = (int)(((int64_t)K + DK - 1) / DK);
  prm.ct = (int)mx_col_tiles(format, K);
  prm.alpha = alpha;
  prm.out = out;
  const int64_t pitch = (int64_t)N * (dtype == FP4MOE_FP32 ? 4 : 2);
  prm.vec = pitch % 32 == 0 && (reinterpret_cast<uintptr_t>(out) & 31u) == 0 ? 5
            : pitch % 16 == 0                                                ? 4
            : pitch % 4 == 0                                                 ? 2
                                                                             : 1;
  prm.err = err;
  const int nsm = sm_count();
  if (nsm <= 0) return FP4MOE_CUDA_ERROR;
  const MxPlan plan = mx_plan(M, N, K, nsm);
  if (plan.pair) return mx_pair_launch(format, dtype, prm, a, a_sf, b, b_sf, st);
  return format == FP4MOE_W_MXFP4 ? dense_width<FP4MOE_W_MXFP4>(plan.bn, dtype, prm, plan.S, a, a_sf, b, b_sf, nsm, st)
                                  : dense_width<FP4MOE_W_NVFP4>(plan.bn, dtype, prm, plan.S, a, a_sf, b, b_sf, nsm, st);
}

}  // namespace fp4moe
