// Dense product of two microscaled 4-bit matrices on CTA pairs: the large sizes of mxdense.cu.
//
// A pair of CTAs owns a 256 x 256 output tile: tcgen05.mma.cta_group::2 of M = 256, N = 256, K = 64, issued by the
// pair's leader (its even CTA), reads 128 rows of A and 128 rows of B from each CTA's shared memory and leaves
// 128 x 256 fp32 in each CTA's TMEM. Against 128 x 256 tiles on single CTAs that halves the B bytes an SM stages
// and reads per MAC: those tiles need 12 KB through shared memory twice (in by TMA, out to the MMA) every 128
// cycles, more than its 128 bytes a cycle.
//   warps 0-7   epilogue, in both CTAs (warp w: TMEM lanes 32 (w % 4) .., columns 128 (w / 4) ..).
//   warp 8      producer, in both CTAs: its own rows of A and B, the scale tiles of its own A rows, and those of all 256
//               B rows (the MMA reads the scales of all 256 B rows from each CTA's own TMEM). All loads signal the
//               leader's barrier. Each CTA loads what it needs itself: the library also runs as replicas on several
//               GPUs, and a load that writes into several CTAs is kept out of it.
//   warp 9      leader: scale copies (tcgen05.cp.cta_group::2, each CTA's tiles into its own TMEM) and MMAs.
// Commits that free a ring stage or hand over the accumulator arrive in both CTAs, and all sixteen epilogue warps tell
// the leader that the accumulator is empty.
//
// 8192 x 4096 x 4096: MXFP4 45.2 us, 6.1 PFLOP/s of the 9.4 that the MMAs reach alone with K = 64, NVFP4 47.8; 8192^3
// 154.6 us, 7.1. The scales of both halves of B are one load of a 3-D map: with a load for each a stage takes 16 ns more
// (46.3, 51.2 and 161 us). What bounds it: a stage of 306 ns, 600 cycles, for MMAs of 512, in which 34 KB enter the SM
// (a quarter fewer of them out of L2 made a stage 5 % faster; five ring stages instead of six 48 us, four 51), and
// 1000 ns between the last MMA of a tile and the first of the next, in which the epilogue empties TMEM: two accumulators
// of 256 columns and the scales do not fit its 512. Not faster: the output by TMA from shared memory (45.0 and 46.9, but
// 8192 x 8192 x 2048 57 instead of 53), all 128 columns of an epilogue warp in flight at once (spills, 53), a stage's
// scale copies ahead of the MMAs before it (50).
// The rest (scale-factor ids, K tails, bounded waits) is as in mxdense.cu.
#include <atomic>

#include "internal.h"
#include "mxdense.cuh"

namespace fp4moe {
namespace {

constexpr int PBM = 256, PBN = 256;  // the pair's tile
constexpr int PEPI = 8;
constexpr int PTHREADS = 32 * (PEPI + 2);
constexpr int PPRODUCER = PEPI, PMMA = PEPI + 1;
constexpr uint32_t PTMEM_COLS = 512;

template <int FMT>
struct PairCfg {
  static constexpr int kSfTiles = FMT == FP4MOE_W_MXFP4 ? 2 : 4;  // scale tiles per 128 rows of a stage
  static constexpr int kA = 128 * 128, kB = 128 * 128;            // this CTA's rows
  static constexpr int kSfa = kSfTiles * 512, kSfb = 2 * kSfa;
  static constexpr int kBytes = kA + kB + kSfa + kSfb;
  static constexpr int kStage = kBytes;
  static constexpr int kStages = FMT == FP4MOE_W_MXFP4 ? 6 : 5;
  static constexpr int kEpiOff = kStages * kStage;  // the epilogue warps' staging areas
  static constexpr int kBarOff = kEpiOff + PEPI * kEpiStage;
  static constexpr int kSmem = kBarOff + 256;  // barriers, and a few words of the CTA
  static constexpr uint32_t kSlotCols = 4 * kSfTiles * 3;
  static_assert(kStage % 1024 == 0, "stage must keep 1024-byte alignment");
  static_assert(PBN + kSlotCols * kStages <= PTMEM_COLS, "accumulator and scale slots fit TMEM");
  static_assert(kSmem <= 232448, "shared memory budget");
  static_assert(8 * (2 * kStages + 3) <= 224, "barriers fit their area");
};

// ------------------------------------------------------------- PTX, CTA pairs
__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const CUtensorMap* map, uint32_t bar, int32_t x,
                                                 int32_t y, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.cta_group::2.L2::cache_hint [%0], "
      "[%1, {%3, %4}], [%2], %5;" ::"r"(dst),
      "l"((uint64_t)map), "r"(bar), "r"(x), "r"(y), "l"(policy)
      : "memory");
}
// Scale tiles [z ..][y ..] of a 3-D map.
__device__ __forceinline__ void tma_load_scales_pair(uint32_t dst, const CUtensorMap* map, uint32_t bar, int32_t y,
                                                     int32_t z, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes.cta_group::2.L2::cache_hint [%0], "
      "[%1, {%3, %4, %5}], [%2], %6;" ::"r"(dst),
      "l"((uint64_t)map), "r"(bar), "r"(0), "r"(y), "r"(z), "l"(policy)
      : "memory");
}
__device__ __forceinline__ void pair_tmem_alloc(uint32_t dst_smem, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_smem), "r"(ncols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void pair_tmem_dealloc(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
// Arrive on this CTA's `bar` once every tcgen05 op this thread issued before has completed in both CTAs.
__device__ __forceinline__ void pair_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
// The same on the barrier at this offset in both CTAs.
__device__ __forceinline__ void pair_commit_both(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
      "h"((uint16_t)3)
      : "memory");
}
__device__ __forceinline__ void pair_cp_scales(uint32_t taddr, uint64_t sdesc) {
  asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(sdesc) : "memory");
}
template <int FMT>
__device__ __forceinline__ void pair_mma(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t sfa,
                                         uint32_t sfb, uint32_t accumulate) {
  if constexpr (FMT == FP4MOE_W_MXFP4)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(
            d),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(
            d),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
}
// A word of another CTA of the cluster (an address from map_cluster), ordered by the cluster's barrier.
__device__ __forceinline__ void st_cluster_u32(uint32_t caddr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(caddr), "r"(v) : "memory");
}
__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t caddr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(caddr) : "memory");
  return v;
}

// Tile t: groups of 4 tile rows, so that the tiles of a wave share their operands' rows in L2 (8192 x 4096 x 4096
// MXFP4 44.7 us; groups of 8 45.0, 16 45.3, 32 46.4).
__device__ __forceinline__ void tile_of(int t, int mt, int nt, int& m, int& n) {
  constexpr int G = 4;
  const int g = t / (G * nt), first = g * G, rows = min(G, mt - first), in = t - g * G * nt;
  m = first + in % rows;
  n = in / rows;
}

template <int FMT, typename T>
__global__ void __launch_bounds__(PTHREADS, 1)
    mx_pair_kernel(const __grid_constant__ DenseMaps maps, const DenseParams prm) {
  using C = PairCfg<FMT>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];  // all of the CTA's shared memory: no static part shifts it
  uint32_t& s_tmem = *reinterpret_cast<uint32_t*>(smem_raw + C::kBarOff + 240);
  uint32_t& s_abort = *reinterpret_cast<uint32_t*>(smem_raw + C::kBarOff + 244);
  // What the CTAs of a pair tell each other at the end: that one gave up (set in both), the ring stages that this CTA's
  // producer has loaded, the stages and tiles that the leader has committed.
  volatile uint32_t* const s_gave_up = reinterpret_cast<uint32_t*>(smem_raw + C::kBarOff + 224);
  volatile int* const s_loaded = reinterpret_cast<int*>(smem_raw + C::kBarOff + 228);
  volatile int* const s_used = reinterpret_cast<int*>(smem_raw + C::kBarOff + 232);
  volatile int* const s_tiles = reinterpret_cast<int*>(smem_raw + C::kBarOff + 236);

  const int warp = __shfl_sync(0xFFFFFFFFu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const uint32_t smem = smem_u32(smem_raw);
  const uint32_t bar_full = smem + C::kBarOff;           // leader's: both CTAs' copies of a stage
  const uint32_t bar_empty = bar_full + 8 * C::kStages;  // each CTA's own: the pair's MMAs have read the stage
  const uint32_t bar_tfull = bar_empty + 8 * C::kStages; // each CTA's own: the accumulator is complete
  const uint32_t bar_tempty = bar_tfull + 8;             // leader's: both CTAs' epilogue warps have read it
  const uint32_t bar_drain = bar_tempty + 8;

  if (warp == 0) pair_tmem_alloc(smem_u32(&s_tmem), PTMEM_COLS);
  if (threadIdx.x == 32 * PPRODUCER) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(bar_full + 8 * s, 1);
      mbar_init(bar_empty + 8 * s, 1);
    }
    mbar_init(bar_tfull, 1);
    mbar_init(bar_tempty, 2 * PEPI);
    mbar_init(bar_drain, 1);
    fence_mbar_init();
  }
  pdl_wait();
  pdl_trigger();
  if (threadIdx.x == 0) {
    s_abort = (*(volatile uint32_t*)prm.err & kAbortMask) != 0 ? 1u : 0u;
    if ((smem & 1023u) != 0) {  // the swizzle needs it, and the compiler grants it
      raise_error(prm.err, FP4MOE_ERR_CAPACITY);
      s_abort = 1u;
    }
    *s_gave_up = 0u;
  }
  tc_fence_before();
  cluster_sync();  // barriers and TMEM of all CTAs are ready
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, s_tmem, 0);
  const int tiles = s_abort ? 0 : prm.mt * prm.nt;  // an earlier timeout poisons the call
  const int KB = prm.KB, pairs = gridDim.x / 2, pair = blockIdx.x / 2;

  const uint32_t far_end = map_cluster(smem + C::kBarOff, rank ^ 1u);  // the words above in the other CTA
  auto give_up = [&]() {
    *s_gave_up = 1u;
    st_cluster_u32(far_end + 224, 1u);
  };
  // this CTA's loads of stage kb of tile (m, n), the it-th that it loads
  const uint32_t full0 = map_cluster(bar_full, 0);
  auto load_stage = [&](int it, int m, int n, int kb, uint64_t pol) {
    const int s = it % C::kStages, ar = 2 * m + (int)rank, br = 2 * n;  // 128-row tiles of A, of B
    const uint32_t st = smem + s * C::kStage, full = full0 + 8 * s, sf = st + C::kA + C::kB;
    if (rank == 0) mbar_arrive_expect_tx(bar_full + 8 * s, 2 * C::kBytes);
    tma_load_2d_pair(st, &maps.a, full, kb * 128, ar * 128, pol);
    tma_load_scales_pair(sf, &maps.sfa, full, kb * C::kSfTiles, ar, pol);
    tma_load_2d_pair(st + C::kA, &maps.b, full, kb * 128, (br + (int)rank) * 128, pol);
    tma_load_scales_pair(sf + C::kSfa, &maps.sfb, full, kb * C::kSfTiles, br, pol);  // rows br and br + 1
  };

  if (warp == PPRODUCER && lane == 0) {
    const uint64_t pol = policy_evict_normal();
    int it = 0;
    bool ok = s_abort == 0;
    for (int t = pair; ok && t < tiles; t += pairs) {
      int m, n;
      tile_of(t, prm.mt, prm.nt, m, n);
      for (int kb = 0; kb < KB; ++kb, ++it) {
        if (!mbar_wait(bar_empty + 8 * (it % C::kStages), ((uint32_t)(it / C::kStages) & 1u) ^ 1u, prm.err)) {
          ok = false;
          break;
        }
        load_stage(it, m, n, kb, pol);
      }
    }
    // the signals that the last stages have been used, and so loaded, are in before the CTA leaves
    for (int j = max(0, it - C::kStages); ok && j < it; ++j)
      ok = mbar_wait(bar_empty + 8 * (j % C::kStages), (uint32_t)(j / C::kStages) & 1u, prm.err);
    *s_loaded = it;
    if (!ok) give_up();
  } else if (warp == PMMA && rank == 0) {
    const bool leader = elect_one();
    int tl = 0, s = 0, used = 0;
    uint32_t ph = 0;
    bool ok = true;
    auto mma = [&](uint64_t adesc, uint64_t bdesc, uint32_t slot, int a, uint32_t acc) {
      constexpr bool mx = FMT == FP4MOE_W_MXFP4;
      const int tile = mx ? a >> 1 : a;
      pair_mma<FMT>(tmem, adesc + 2 * a, bdesc + 2 * a,
                    idesc_mx<FMT>(PBM, PBN, mx ? 2 * (a & 1) : 0), slot + 4 * tile, slot + 4 * C::kSfTiles + 8 * tile,
                    acc);
    };
    for (int t = pair; t < tiles; t += pairs, ++tl) {
      // both epilogues have moved the previous tile's accumulator out of TMEM
      const uint32_t tph = ((uint32_t)tl & 1u) ^ 1u;
      ok = mbar_wait_warp(bar_tempty, tph, prm.err);
      if (!ok) break;
      tc_fence_after();
      for (int kb = 0; kb < KB; ++kb, ++used) {
        if (!mbar_wait_warp(bar_full + 8 * s, ph, prm.err)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t st = smem + (uint32_t)s * C::kStage, slot = tmem + PBN + C::kSlotCols * s;
        const int atoms = (prm.K - kb * DK + 63) / 64;  // of this stage and those behind it
        if (leader) {
          // A tile i, then B tile j half h at column 4 (2 j + h): an N = 256 MMA takes the two halves side by side.
          // Copies and MMAs of one thread execute in order, and slot s is free: its last MMAs committed bar_empty.
          // Descriptors hold addresses in units of 16 bytes; within a stage they are added to.
          const uint64_t ad = desc_sw128(st), bd = desc_sw128(st + C::kA), sd = desc_scales(st + C::kA + C::kB);
#pragma unroll
          for (int i = 0; i < C::kSfTiles; ++i) pair_cp_scales(slot + 4 * i, sd + 32 * i);
#pragma unroll
          for (int j = 0; j < C::kSfTiles; ++j)
#pragma unroll
            for (int h = 0; h < 2; ++h)
              pair_cp_scales(slot + 4 * C::kSfTiles + 4 * (2 * j + h), sd + C::kSfa / 16 * (1 + h) + 32 * j);
          if (atoms >= 4) {
#pragma unroll
            for (int a = 0; a < 4; ++a) mma(ad, bd, slot, a, (kb > 0 || a > 0) ? 1u : 0u);
          } else {
#pragma unroll
            for (int a = 0; a < 3; ++a)
              if (a < atoms) mma(ad, bd, slot, a, (kb > 0 || a > 0) ? 1u : 0u);
          }
          pair_commit_both(bar_empty + 8 * s);
        }
        __syncwarp();
        if (++s == C::kStages) {
          s = 0;
          ph ^= 1u;
        }
      }
      if (!ok) break;
      if (leader) pair_commit_both(bar_tfull);
    }
    if (leader) {
      *s_used = used;
      *s_tiles = tl;
      if (!ok) give_up();
      pair_commit(bar_drain);
      drain_wait(bar_drain, 0);  // no MMA may still write TMEM when it is freed
    }
  } else if (warp < PEPI) {
    constexpr int W = PBN / 2;  // columns of one warp
    const int quarter = warp & 3, half = warp >> 2;
    uint8_t* stage = smem_raw + C::kEpiOff + warp * kEpiStage;
    // Arrivals here publish no memory writes: what they order are TMEM reads, complete at the arriving warp's
    // tcgen05.wait::ld, with the tcgen05 fences of both sides. A release at cluster scope and a fence at the other end
    // cost 1.1 us a tile.
    const uint32_t tempty = map_cluster(bar_tempty, 0);
    const float alpha = prm.alpha != nullptr ? __ldg(prm.alpha) : 1.0f;
    int tl = 0;
    for (int t = pair; t < tiles; t += pairs, ++tl) {
      int m, n;
      tile_of(t, prm.mt, prm.nt, m, n);
      const int r0 = m * PBM + (int)rank * 128 + quarter * 32;
      const int c0 = n * PBN + W * half;
      // the whole warp takes one decision: tcgen05.ld is warp-collective
      if (!mbar_wait_warp(bar_tfull, (uint32_t)tl & 1u, prm.err)) {
        if (lane == 0) give_up();
        break;
      }
      tc_fence_after();
      const bool live = r0 < prm.M && c0 < prm.N;
      uint32_t w[W * sizeof(T) / 4];
      if (live) load_packed<T, W>(tmem + (uint32_t)(W * half) + ((uint32_t)(quarter * 32) << 16), alpha, w);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(tempty);  // this warp's share of the accumulator is out of TMEM
      if (live) {
        constexpr int COLS = 64 / (int)sizeof(T);
#pragma unroll
        for (int c = 0; c < W; c += COLS)
          if (c0 + c < prm.N)
            store_chunk(stage, w + c * (int)sizeof(T) / 4, static_cast<T*>(prm.out), prm.M, prm.N, r0, c0 + c, lane,
                        prm.vec);
      }
    }
  }
  __syncwarp();  // the single-thread roles reconverge: cluster barriers are warp-aligned instructions
  tc_fence_before();
  cluster_sync();  // no CTA reads or signals another any more, unless one gave up
  if (*s_gave_up != 0) {
    // All that is in flight lands before either CTA leaves. The leader's barrier for a stage counts the loads of both
    // CTAs, so the one whose producer stopped first loads what the other has loaded already (into stages that no MMA
    // reads any more, at most a ring's worth); and commits signal both CTAs.
    if (warp == PPRODUCER && lane == 0) {
      const int other = (int)ld_cluster_u32(far_end + 228);
      const int mine = *s_loaded, loaded = max(mine, other);
      for (int j = mine; j < loaded; ++j) {
        int m, n;
        tile_of(pair + j / KB * pairs, prm.mt, prm.nt, m, n);
        load_stage(j, m, n, j % KB, policy_evict_normal());
      }
      if (rank == 0) {
        for (int j = max(0, loaded - C::kStages); j < loaded; ++j)
          drain_wait(bar_full + 8 * (j % C::kStages), (uint32_t)(j / C::kStages) & 1u);
      }
      const int used = rank == 0 ? *s_used : (int)ld_cluster_u32(far_end + 232);
      const int done = rank == 0 ? *s_tiles : (int)ld_cluster_u32(far_end + 236);
      for (int j = max(0, used - C::kStages); j < used; ++j)
        drain_wait(bar_empty + 8 * (j % C::kStages), (uint32_t)(j / C::kStages) & 1u);
      if (done > 0) drain_wait(bar_tfull, (uint32_t)(done - 1) & 1u);
    }
    __syncwarp();
    cluster_sync();
  }
  if (warp == 0) {
    tc_fence_after();
    pair_tmem_dealloc(tmem, PTMEM_COLS);
  }
}

// The driver's cuTensorMapEncodeTiled, reached at run time: the library loads where there is no driver.
decltype(&cuTensorMapEncodeTiled) tiled_encoder() {
  static std::atomic<void*> known{nullptr};
  void* p = known.load(std::memory_order_acquire);
  if (p == nullptr) {
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return nullptr;
    known.store(p, std::memory_order_release);
  }
  return reinterpret_cast<decltype(&cuTensorMapEncodeTiled)>(p);
}

// Scale tiles (512 bytes each) as a 3-D tensor [row_tiles][col_tiles][128 words], unswizzled boxes of
// box_rows x box_cols whole tiles.
bool encode_scale_tiles(CUtensorMap* m, const void* base, uint64_t row_tiles, uint64_t col_tiles, uint32_t box_rows,
                        uint32_t box_cols) {
  const auto encode = tiled_encoder();
  if (encode == nullptr) return false;
  const cuuint64_t dims[3] = {128, col_tiles, row_tiles}, strides[2] = {512, 512 * col_tiles};
  const cuuint32_t box[3] = {128, box_cols, box_rows}, es[3] = {1, 1, 1};
  return encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT32, 3, const_cast<void*>(base), dims, strides, box, es,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The cluster shape's launch attributes; PDL as in launch_pdl.
cudaLaunchConfig_t pair_config(unsigned pairs, size_t smem, cudaStream_t st, cudaLaunchAttribute (&attr)[2]) {
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3(2u * pairs);
  lc.blockDim = dim3(PTHREADS);
  lc.dynamicSmemBytes = smem;
  lc.stream = st;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = attr;
  lc.numAttrs = 2;
  return lc;
}

// Pairs that the device holds at once (the persistent grid); 0 on error. Kept for each device.
template <int FMT, typename T>
int pair_count() {
  static PerDevice count;
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  return count.get(dev, [] {
    int n = 0;
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t lc = pair_config(1, PairCfg<FMT>::kSmem, nullptr, attr);
    lc.numAttrs = 1;  // the cluster shape alone
    if (cudaFuncSetAttribute(mx_pair_kernel<FMT, T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             PairCfg<FMT>::kSmem) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, mx_pair_kernel<FMT, T>, &lc) != cudaSuccess)
      n = 0;
    return n;
  });
}

template <int FMT, typename T>
fp4moe_status pair_run(DenseParams prm, const uint8_t* a, const uint8_t* a_sf, const uint8_t* b, const uint8_t* b_sf,
                       cudaStream_t st) {
  using C = PairCfg<FMT>;
  prm.mt = (prm.M + PBM - 1) / PBM;
  prm.nt = (prm.N + PBN - 1) / PBN;
  DenseMaps maps;
  const uint64_t rb = (uint64_t)mx_row_bytes(prm.K);
  if (!encode_u8_sw128(&maps.a, a, rb, (uint64_t)prm.M, 128) ||
      !encode_u8_sw128(&maps.b, b, rb, (uint64_t)prm.N, 128) ||
      !encode_scale_tiles(&maps.sfa, a_sf, (uint64_t)mx_row_tiles(prm.M), (uint64_t)prm.ct, 1, C::kSfTiles) ||
      !encode_scale_tiles(&maps.sfb, b_sf, (uint64_t)mx_row_tiles(prm.N), (uint64_t)prm.ct, 2, C::kSfTiles))
    return FP4MOE_CUDA_ERROR;
  const int most = pair_count<FMT, T>(), tiles = prm.mt * prm.nt;
  if (most <= 0) return FP4MOE_CUDA_ERROR;
  cudaLaunchAttribute attr[2];
  const cudaLaunchConfig_t lc = pair_config((unsigned)(tiles < most ? tiles : most), C::kSmem, st, attr);
  return cudaLaunchKernelEx(&lc, mx_pair_kernel<FMT, T>, maps, prm) == cudaSuccess ? FP4MOE_OK
                                                                                        : FP4MOE_CUDA_ERROR;
}

template <int FMT>
fp4moe_status pair_typed(int32_t dtype, const DenseParams& prm, const uint8_t* a, const uint8_t* a_sf,
                         const uint8_t* b, const uint8_t* b_sf, cudaStream_t st) {
  switch (dtype) {
    case FP4MOE_BF16:
      return pair_run<FMT, __nv_bfloat16>(prm, a, a_sf, b, b_sf, st);
    case FP4MOE_FP16:
      return pair_run<FMT, __half>(prm, a, a_sf, b, b_sf, st);
    default:
      return pair_run<FMT, float>(prm, a, a_sf, b, b_sf, st);
  }
}

}  // namespace

fp4moe_status mx_pair_launch(int32_t format, int32_t dtype, const DenseParams& prm, const uint8_t* a,
                             const uint8_t* a_sf, const uint8_t* b, const uint8_t* b_sf, cudaStream_t st) {
  return format == FP4MOE_W_MXFP4 ? pair_typed<FP4MOE_W_MXFP4>(dtype, prm, a, a_sf, b, b_sf, st)
                                  : pair_typed<FP4MOE_W_NVFP4>(dtype, prm, a, a_sf, b, b_sf, st);
}

}  // namespace fp4moe
