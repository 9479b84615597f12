// Attention over the paged cache for many rows a sequence and kv head (fp4moe_paged_attention): prompts and chunks of them.
//
// A unit is 256 rows, as two tiles of 128, against its keys in steps of 128:
//   S = Q K^T          tcgen05.mma, M = 128, N = 128: Q and K in shared memory, S (fp32) in TMEM
//   P = 2^(S - m)      one thread a row: S out of TMEM, P (16 bits) back into the place of S
//   O += P V           tcgen05.mma with P out of TMEM, V in shared memory as it lies (keys x dims: transposed B), O in TMEM
// The tensor cores work on one tile while the other's softmax runs:
//   warps 0-3, 4-7     softmax, rescaling and output of tile 0 and 1 (warp w: TMEM lanes 32 (w % 4) ..)
//   warp 8             MMAs of both tiles in turn: for each step the P V of the step before and the next Q K^T
//   warp 9, warp 10    loads of q and k, and of v, into 128-byte-swizzled tiles. By TMA where pages consist of whole 8-row
//                      swizzle atoms: a box is 64 dims of the keys that a page and a step share (gcd(page size, 128)), one
//                      lane a box. Other page sizes by gathers of four rows where all slots lie evenly apart and heads
//                      are whole MMA steps, one lane a gather, else by 16-byte cp.async, a lane looking a key's place up for the lanes that copy it.
// The MMAs of a tile come from one thread and run in order, so a finished S(j) means a finished P V(j - 1): O may be rescaled then, and P(j) may
// take the place of S(j). P is made under the maximum of the steps before, so that finding this step's is not in its way;
// only where that had grown by more than 2^8 is O rescaled and P made again (weights up to 2^8, in fp16 2^15: attn.cuh).
// Scores of keys that a row does not see are -infinity; v of keys outside the tile's range is zeroed in shared memory, for 0
// times what lies there may be NaN. So does what is not finite of a v that only some rows of the unit see: those add weight
// times it in the end. Such keys lie at the ends of a unit's range, at most 2 x 255 of them, however long it is.
// Every wait is bounded, as in the layer's GEMMs.
//
// What bounds it: a tile's round from its scores to its weights to the next scores, 3000 cycles, in which the MMAs of both
// tiles take 2064 (128 dims); a third tile has no room in TMEM. A causal prompt of 8192 tokens, 32 / 8 heads of 128 dims: 388
// us, 1417 TFLOP/s, for twenty calls one after the other, 406 over seconds, plain or in a graph, when the power limit takes the
// clock from 2070 to 1970 MHz; chunks of 512 tokens behind up to 3584, eight sequences: 132 us, 1010 TFLOP/s, of which 5 us begin
// and end a CTA's run. Measured on the prompt: one warp for the MMAs of both tiles 406 and one each 489 (the tiles fall into
// step); weights under the maximum so far 448 and under the new one 483; one lane of a converged warp issues MMAs 483 and a
// lane picked by index 573; boxes 1056 and cp.async 1206. Chunks over pages of one token: gathers 207, cp.async 438.
#include "attn.cuh"
#include "inflight.h"

namespace fp4moe {
namespace {

constexpr int AT_BM = 256, AT_KEYS = 128;
constexpr int AT_ODD = 8;          // units whose flags are kept: loads run ahead by a unit for each stage at most
constexpr int AT_FEW = 32;         // rows of a tile whose parts are joined a few lanes a row
constexpr int AT_MIN = 4;          // least cost of a CTA's run
constexpr int AT_OH = 4;           // what a unit costs, in steps, beside its steps
constexpr int AT_THREADS = 352;    // 168 registers a thread, for a row of S; 80 to 88 bytes beside it are spilled
constexpr float AT_GROWTH = 8.0f;  // powers of two that a maximum may lag behind

template <int DP>
struct TileCfg {
  static constexpr int kBlocks = DP / 64;             // 128-byte columns of a tile
  static constexpr int kBlock = 128 * 128;            // bytes of 128 rows of one
  static constexpr int kTile = kBlocks * kBlock;      // 128 rows of q, k or v
  static constexpr int kStages = DP == 128 ? 2 : 4;   // of k, and of v
  static constexpr int kK = 2 * kTile, kV = kK + kStages * kTile;
  static constexpr int kBars = kV + kStages * kTile;
  static constexpr int kOut = kBars + 512;            // the softmax warps' output, 32 rows x 32 dims each
  static constexpr int kSmem = kOut + 8 * 2048 + 1024;  // and to align it
  static_assert(kSmem <= 232448, "shared memory budget");
  static_assert(AT_ODD > kStages + 1, "a unit's flag is read before it is another's");
  static_assert((FP4MOE_KV_MAX_SEQS + AT_THREADS / 32 + 1) * 8 <= kBars, "the division's sums fit");
};

// Barriers, 8 bytes each, behind the tiles.
template <int DP>
struct TileBars {
  using C = TileCfg<DP>;
  uint32_t base;
  __device__ __forceinline__ uint32_t k_full(int s) const { return base + 8 * s; }
  __device__ __forceinline__ uint32_t k_empty(int s) const { return base + 8 * (C::kStages + s); }
  __device__ __forceinline__ uint32_t v_full(int s) const { return base + 8 * (2 * C::kStages + s); }
  __device__ __forceinline__ uint32_t v_empty(int s) const { return base + 8 * (3 * C::kStages + s); }
  __device__ __forceinline__ uint32_t q_full() const { return base + 8 * (4 * C::kStages); }
  __device__ __forceinline__ uint32_t q_empty() const { return base + 8 * (4 * C::kStages + 1); }
  __device__ __forceinline__ uint32_t s_full(int t) const { return base + 8 * (4 * C::kStages + 2 + t); }
  __device__ __forceinline__ uint32_t p_full(int t) const { return base + 8 * (4 * C::kStages + 4 + t); }
  __device__ __forceinline__ uint32_t o_full(int t) const { return base + 8 * (4 * C::kStages + 6 + t); }
  __device__ __forceinline__ uint32_t join(int t) const { return base + 8 * (4 * C::kStages + 8 + t); }
  __device__ __forceinline__ uint32_t done() const { return base + 8 * (4 * C::kStages + 10); }
  __device__ __forceinline__ uint32_t landed() const { return base + 8 * (4 * C::kStages + 11); }
};

// Tensor maps: k and v as [pages][tokens][heads][dims], boxes of `rows` tokens x 64 dims; q as [T][heads][dims], boxes of
// 128 rows x 64 dims where the heads of a group divide 128.
struct TileMaps {
  CUtensorMap k, v, q;
  int rows;   // of a box; 1: four rows at a time, wherever they lie (k and v as [slots][heads and dims]); 0: no boxes, by cp.async
  int q_box;  // whether q has boxes
};
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y, int z, int w) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(
          dst),
      "l"((uint64_t)map), "r"(bar), "r"(x), "r"(y), "r"(z), "r"(w)
      : "memory");
}
__device__ __forceinline__ void tma_gather4(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, const int (&row)[4]) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6, "
      "%7}], [%2];" ::"r"(dst),
      "l"((uint64_t)map), "r"(bar), "r"(x), "r"(row[0]), "r"(row[1]), "r"(row[2]), "r"(row[3])
      : "memory");
}
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"((uint64_t)map), "r"(bar), "r"(x), "r"(y), "r"(z)
      : "memory");
}

// Whether the phase has completed, without waiting (try_wait may suspend the thread for microseconds).
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
// One lane of a converged warp, which the compiler knows to be one: descriptors stay in uniform registers, where the MMA
// wants them (a lane picked by its index costs several register moves an MMA).
__device__ __forceinline__ bool elect_one() {
  uint32_t ok;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(ok));
  return ok != 0;
}
// The whole warp waits, and goes on together.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, uint32_t* err) {
  return __all_sync(0xFFFFFFFFu, mbar_wait(bar, parity, err));
}

// A (K-major) and B: both bf16 or both fp16, fp32 D; transposed B: stored K x N with N contiguous.
template <typename T>
__device__ __forceinline__ constexpr uint32_t idesc_16(int N, bool transposed_b) {
  constexpr uint32_t F = std::is_same_v<T, __nv_bfloat16> ? 1u : 0u;
  return (1u << 4) | (F << 7) | (F << 10) | ((transposed_b ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) | ((128u >> 4) << 24);
}
// Descriptor of a transposed B tile: 64 columns (128 swizzled bytes) a row, 8 rows 1024 bytes, the next 64 columns
// `block` bytes on.
__device__ __forceinline__ uint64_t desc_sw128_t(uint32_t saddr, uint32_t block) {
  return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)(block >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
         ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  tc_mma_bf16(d, a, b, idesc, accumulate);  // (kind::f16 is both types; idesc says which)
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]),
      "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
      "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(taddr)
      : "memory");
}
// The loads of v, and whatever was loaded before, have arrived: nothing may use v earlier.
__device__ __forceinline__ void tmem_arrived(float (&v)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]), "+f"(v[8]),
                 "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15]), "+f"(v[16]),
                 "+f"(v[17]), "+f"(v[18]), "+f"(v[19]), "+f"(v[20]), "+f"(v[21]), "+f"(v[22]), "+f"(v[23]), "+f"(v[24]),
                 "+f"(v[25]), "+f"(v[26]), "+f"(v[27]), "+f"(v[28])
               :
               : "memory");
  asm volatile("" : "+f"(v[29]), "+f"(v[30]), "+f"(v[31]) : : "memory");
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// Two of each in one instruction.
__device__ __forceinline__ void fma2(float& x, float& y, float a, float b, float f, float c) {  // (x, y) = (a, b) f + c
  asm("{\n\t.reg .b64 u, v, w;\n\tmov.b64 u, {%2, %3};\n\tmov.b64 v, {%4, %4};\n\tmov.b64 w, {%5, %5};\n\t"
      "fma.rn.f32x2 u, u, v, w;\n\tmov.b64 {%0, %1}, u;\n\t}"
      : "=f"(x), "=f"(y)
      : "f"(a), "f"(b), "f"(f), "f"(c));
}
__device__ __forceinline__ void add2(float& x, float& y, float a, float b) {  // (x, y) += (a, b)
  asm("{\n\t.reg .b64 u, v;\n\tmov.b64 u, {%0, %1};\n\tmov.b64 v, {%2, %3};\n\tadd.rn.f32x2 u, u, v;\n\t"
      "mov.b64 {%0, %1}, u;\n\t}"
      : "+f"(x), "+f"(y)
      : "f"(a), "f"(b));
}
// 8 columns in and out, times f: few registers beside a row of S.
__device__ __forceinline__ void tmem_scale8(uint32_t taddr, float f) {
  uint32_t r[8];
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr)
               : "memory");
  tmem_ld_wait();
#pragma unroll
  for (int c = 0; c < 8; ++c) r[c] = __float_as_uint(__uint_as_float(r[c]) * f);
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0,%1,%2,%3,%4,%5,%6,%7};" ::"r"(r[0]), "r"(r[1]), "r"(r[2]),
               "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(taddr)
               : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// ---------------------------------------------------------------- loads (one warp for q and k, one for v)
template <typename T, int DP>
struct Loader {
  using C = TileCfg<DP>;
  static constexpr int CH = DP / 8, RPI = 32 / CH;  // 16-byte pieces of a row; rows of a warp's copy instruction
  const AttnParams& p;
  const TileBars<DP>& bar;
  uint32_t sm32;
  int lane, dims;
  // 32 rows from row0 on; `off` is the element offset of this lane's row, negative: zeros.
  __device__ __forceinline__ void rows32(uint32_t tile, int row0, const T* base, int64_t off) {
    const int c = lane % CH;
#pragma unroll
    for (int it = 0; it < 32 / RPI; ++it) {
      const int r = it * RPI + lane / CH;
      const int64_t ro = __shfl_sync(0xFFFFFFFFu, off, r);
      const bool use = ro >= 0 && c * 8 < p.D;
      const int row = row0 + r;
      if (c * 8 < dims)
        cp_async16(tile + (c >> 3) * C::kBlock + row * 128 + (((c & 7) ^ (row & 7)) << 4), base + (use ? ro + c * 8 : 0), use);
    }
  }
  // All copies issued so far have landed: tell it.
  __device__ __forceinline__ void told(uint32_t b) {
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(b);
  }
  // One tile (128 rows) of the unit's q, by cp.async.
  __device__ __forceinline__ void q_rows(const AttnUnit& u, int t) {
#pragma unroll 1
    for (int r0 = 0; r0 < 128; r0 += 32) {
      const int r = t * 128 + r0 + lane;
      int64_t off = -1;
      if (r < u.rows) {
        const int tok = (int)p.group.div(u.row0 + r), g = u.row0 + r - tok * (int)p.group.d;
        off = (int64_t)(u.seq.first + tok) * p.q_stride + (int64_t)(u.head * (int)p.group.d + g) * p.D;
      }
      rows32(sm32 + t * C::kTile, r0, static_cast<const T*>(p.q), off);
    }
    cp_async_commit();
    cp_async_wait<0>();
    told(bar.q_full());
  }
  // Where a key of the unit lies: its page, or num_pages (zeros) if it has none or a bad one.
  __device__ __forceinline__ int page_of(const AttnUnit& u, const int32_t* table, int key, bool there) {
    return there && key >= u.range.x && key < u.range.y ? table[p.map.page.div(key)] : -2;
  }
  __device__ __forceinline__ int checked(int page) {
    if ((uint32_t)page < (uint32_t)p.map.num_pages) return page;
    if (page != -2) raise_error(p.err, FP4MOE_ERR_PAGE);
    return p.map.num_pages;
  }
  __device__ __forceinline__ int in_page(int key) { return key - (int)p.map.page.div(key) * (int)p.map.page.d; }
  // 128 keys from k0 on into `tile`, by cp.async; page[h]: that of key k0 + 32 h + lane.
  __device__ __forceinline__ void key_rows(const AttnUnit& u, uint32_t tile, const T* base, int k0, const int (&page)[4]) {
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      const int pg = checked(page[h]);
      const int64_t off = pg == p.map.num_pages ? -1
                                                : pg * p.map.page_stride + (int64_t)in_page(k0 + h * 32 + lane) * p.map.token_stride +
                                                      (int64_t)u.head * p.map.head_stride;
      rows32(tile, h * 32, base, off);
    }
    cp_async_commit();
  }
};

// Zeros for what is not finite in rows [lo, hi) of a tile of v but [all_lo, all_hi), by a warp. (rare: kept out of the loads)
template <typename T, int DP>
__device__ __noinline__ void keep_finite(uint8_t* tile, int lo, int all_lo, int all_hi, int hi) {
  using C = TileCfg<DP>;
  constexpr int PER = C::kBlocks * 8;  // 16-byte pieces of a row
  constexpr uint32_t E = std::is_same_v<T, __nv_bfloat16> ? 0x7F80u : 0x7C00u;
  for (int i = max(lo, 0) * PER + (int)lane_id(); i < min(hi, 128) * PER; i += 32) {
    const int row = i / PER, c = i % PER;
    if (row >= all_lo && row < all_hi) continue;
    uint4* at = reinterpret_cast<uint4*>(tile + (c >> 3) * C::kBlock + row * 128 + (((c & 7) ^ (row & 7)) << 4));
    uint32_t w[4] = {at->x, at->y, at->z, at->w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if ((w[e] & E) == E) w[e] &= 0xFFFF0000u;
      if (((w[e] >> 16) & E) == E) w[e] &= 0xFFFFu;
    }
    *at = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// How k and v are brought: by cp.async, by boxes of a page's keys, or by gathers of four keys a lane.
enum LoadMode { kCopies = 0, kBoxes = 1, kGathers = 2 };
// One of the two streams: WHICH = 0 k (and q), 1 v. Stages go round; load n is told on full(n % kStages).
template <typename T, int DP, int MODE, int WHICH>
__device__ __forceinline__ void load_role(const AttnParams& p, const TileMaps& maps, const AttnRun& run, const TileBars<DP>& bar,
                                          uint8_t* sm, uint32_t sm32, volatile int* odd) {
  using C = TileCfg<DP>;
  const int lane = lane_id();
  Loader<T, DP> L{p, bar, sm32, lane, (p.D + 15) / 16 * 16};
  const T* base = static_cast<const T*>(WHICH ? p.v : p.k);
  const CUtensorMap* map = WHICH ? &maps.v : &maps.k;
  const uint32_t tiles = WHICH ? C::kV : C::kK;
  auto full = [&](int s) { return WHICH ? bar.v_full(s) : bar.k_full(s); };
  auto empty = [&](int s) { return WHICH ? bar.v_empty(s) : bar.k_empty(s); };
  constexpr bool BOXES = MODE != kCopies, gather = MODE == kGathers;
  const int per = !BOXES ? 1 : gather ? 32 : 128 / maps.rows, boxes = per * (p.D > 64 ? 2 : 1);  // of a step: one lane each
  const int box_key = lane % per * maps.rows, box_col = lane / per;
  int stage = 0, units = 0;
  uint32_t phase = 0;
  int64_t issued = 0;
  InFlight q_boxes;  // loads of q on q_full
  bool ok = true;
  // The load that is looked after once it has landed: a step of v that is not all visible to all rows, or one by cp.async.
  struct {
    bool any, rows;  // rows: zero those outside [lo, hi); mark: unit + 1 if those that not all rows see are looked through
    int stage, k0, lo, hi, all_lo, all_hi, mark;
    int64_t n;
  } late{};
  uint32_t landed = 0;
  auto look_after = [&](bool newer) -> bool {  // newer: a cp.async load has been issued since
    if (!late.any) return true;
    if (BOXES) {
      if (!warp_wait(bar.landed(), landed, p.err)) return false;
      landed ^= 1;
    } else {
      if (newer) cp_async_wait<1>();
      else cp_async_wait<0>();
      __syncwarp();
    }
    late.any = false;
    if (WHICH && (late.rows || late.mark)) {
      bool bad = false;
      uint8_t* tile = sm + C::kV + late.stage * C::kTile;
      constexpr int PER = C::kBlocks * 8;  // 16-byte pieces of a row
      auto piece = [&](int i) {
        const int row = i / PER, c = i % PER;
        return reinterpret_cast<uint4*>(tile + (c >> 3) * C::kBlock + row * 128 + (((c & 7) ^ (row & 7)) << 4));
      };
      if (late.rows) {
        const int lo = max(late.lo - late.k0, 0) * PER, hi = min(max(late.hi - late.k0, 0), 128) * PER;
        for (int i = lane; i < lo; i += 32) *piece(i) = make_uint4(0u, 0u, 0u, 0u);
        for (int i = hi + lane; i < 128 * PER; i += 32) *piece(i) = make_uint4(0u, 0u, 0u, 0u);
        __syncwarp();
      }
      if (late.mark) {
        auto look = [&](int from, int to) {
          from = max(from - late.k0, 0) * PER;
          to = min(to - late.k0, 128) * PER;
#pragma unroll 4
          for (int i = lane % PER * 8 < p.D ? from + lane : to; i < to; i += 32)  // (past the head's dims lies anything)
            bad |= any_nonfinite<T>(*piece(i));
        };
        if (late.all_lo < late.all_hi) {
          look(late.lo, late.all_lo);
          look(late.all_hi, late.hi);
        } else {
          look(late.lo, late.hi);
        }
      }
      if (__any_sync(0xFFFFFFFFu, bad)) {
        keep_finite<T, DP>(tile, late.lo - late.k0, late.all_lo - late.k0, late.all_hi - late.k0, late.hi - late.k0);
        odd[(late.mark - 1) % AT_ODD] = late.mark;
      }
    }
    L.told(full(late.stage));
    return true;
  };
  AttnWalk walk(run);
  for (AttnUnit u; ok && walk.next<AT_BM, AT_KEYS, AT_OH>(p, run, u); ++units) {
    const int n = u.s1 - u.s0, first = (u.range.x / AT_KEYS + u.s0) * AT_KEYS;
    const int32_t* table = p.table + (int64_t)u.b * p.columns;
    int page[4];
    auto look_up = [&](int i) {
      const int k0 = first + i * AT_KEYS;
      if constexpr (gather) {
#pragma unroll
        for (int h = 0; h < 4; ++h) page[h] = L.page_of(u, table, k0 + lane * 4 + h, i < n);
      } else if constexpr (BOXES) {
        page[0] = L.page_of(u, table, max(k0 + box_key, u.range.x), i < n && lane < boxes && k0 + box_key + maps.rows > u.range.x);
      } else {
#pragma unroll
        for (int h = 0; h < 4; ++h) page[h] = L.page_of(u, table, k0 + h * 32 + lane, i < n);
      }
    };
    look_up(0);
    if (WHICH == 0 || !maps.q_box) {
      if (!(ok = warp_wait(bar.q_empty(), (units & 1) ^ 1, p.err))) break;
      const int qt = u.rows > 128 ? 2 : 1;
      if (!maps.q_box) {
        L.q_rows(u, WHICH);
      } else {
        const int blocks = p.D > 64 ? 2 : 1;
        if (lane == 0) mbar_arrive_expect_tx(bar.q_full(), qt * blocks * C::kBlock);
        __syncwarp();
        q_boxes.issue();
        if (lane < qt * blocks) {
          const int t = lane / blocks, b = lane % blocks;
          tma_load_3d(sm32 + t * C::kTile + b * C::kBlock, &maps.q, bar.q_full(), b * 64, u.head * (int)p.group.d,
                      u.seq.first + (int)p.group.div(u.row0 + t * 128));
        }
      }
    }
    const int all_lo = attn_range(p, u.seq, u.kv, (int)p.group.div(u.row0 + u.rows - 1)).x;
    const int all_hi = attn_range(p, u.seq, u.kv, (int)p.group.div(u.row0)).y;
    for (int i = 0; i < n; ++i) {
      const int k0 = first + i * AT_KEYS;
      const bool edge = k0 < u.range.x || k0 + AT_KEYS > u.range.y, some = k0 < all_lo || k0 + AT_KEYS > all_hi;
      const bool differ = some && (all_lo != u.range.x || all_hi != u.range.y);
      const bool look = !BOXES || (WHICH && (edge || differ));
      const uint32_t tile = sm32 + tiles + stage * C::kTile, b = BOXES && look ? bar.landed() : full(stage);
      int box_tok = 0, box_page = 0, slot[4];
      if constexpr (gather) {  // (a row past the last reads as zeros)
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          const int pg = L.checked(page[h]);
          slot[h] = pg * (int)p.map.page.d + (pg == p.map.num_pages ? 0 : L.in_page(k0 + lane * 4 + h));
        }
      } else if constexpr (BOXES) {
        box_tok = L.in_page(k0 + box_key);
        box_page = L.checked(page[0]);
      }
      if (BOXES && look && !(ok = look_after(false))) break;  // one at a time
      // what is late may be what frees the stage
      if (late.any && !mbar_test(empty(stage), phase ^ 1) && !(ok = look_after(false))) break;
      if (!(ok = warp_wait(empty(stage), phase ^ 1, p.err))) break;
      if (BOXES) {
        if (lane == 0) mbar_arrive_expect_tx(b, (p.D > 64 ? 2 : 1) * C::kBlock);
        __syncwarp();
        if constexpr (gather) {
          const int x = u.head * (int)p.map.head_stride;
          for (int c = 0; c < (p.D > 64 ? 2 : 1); ++c) tma_gather4(tile + c * C::kBlock + lane * 512, map, b, x + c * 64, slot);
        } else if (lane < boxes) {
          tma_load_4d(tile + box_col * C::kBlock + box_key * 128, map, b, box_col * 64, u.head, box_tok, box_page);
        }
      } else {
        L.key_rows(u, tile, base, k0, page);
      }
      look_up(i + 1);
      if (!BOXES && !(ok = look_after(true))) break;
      if (look) {
        late.any = true;
        late.rows = BOXES && edge;  // (cp.async has filled them with zeros)
        late.stage = stage;
        late.k0 = k0;
        late.lo = u.range.x;
        late.hi = u.range.y;
        late.all_lo = all_lo;
        late.all_hi = all_hi;
        late.mark = differ ? units + 1 : 0;
        late.n = issued;
      }
      ++issued;
      if (++stage == C::kStages) {
        stage = 0;
        phase ^= 1;
      }
    }
    if (ok) ok = look_after(false);
  }
  cp_async_wait<0>();
  if (BOXES && !ok) {  // it gave up: what is in flight still has to land
    if (late.any) drain_wait(bar.landed(), landed);
    for (int64_t i = issued > C::kStages ? issued - C::kStages : 0; i < issued; ++i)
      if (!late.any || i != late.n) drain_wait(full(i % C::kStages), (i / C::kStages) & 1);
  }
  if (!ok && q_boxes.any()) drain_wait(bar.q_full(), q_boxes.last());
}

// ---------------------------------------------------------------- MMAs (one warp)
template <typename T, int DP>
__device__ __forceinline__ void mma_role(const AttnParams& p, const AttnRun& run, const TileBars<DP>& bar, uint32_t sm32,
                                         uint32_t tmem) {
  using C = TileCfg<DP>;
  const int dims = (p.D + 15) / 16 * 16;
  const uint32_t is = idesc_16<T>(AT_KEYS, false), io = idesc_16<T>(dims, true);
  int ks = 0, vs = 0, units = 0;
  uint32_t kp = 0, vp = 0, pp[2] = {0, 0};  // phases of the k and v stages, and of the p barriers
  // descriptors count in 16 bytes, so offsets are added to them
  const uint64_t qd = desc_sw128(sm32), kd = desc_sw128(sm32 + C::kK), vd = desc_sw128_t(sm32 + C::kV, C::kBlock);
  // A wait that gave up is only looked at once a step: what is issued until then reads and writes this CTA's own memory.
  bool ok = true;
  auto wait = [&](uint32_t b, uint32_t parity) { ok &= mbar_wait(b, parity, p.err); };
  const bool leader = elect_one();
  AttnWalk walk(run);
  for (AttnUnit u; ok && walk.next<AT_BM, AT_KEYS, AT_OH>(p, run, u); ++units) {
    const bool two = u.rows > 128;
    const int n = u.s1 - u.s0;
    wait(bar.q_full(), units & 1);
    bool k_there = false, v_there = false;  // the next step's, known already
    for (int j = 0; j <= n; ++j) {
      if (!k_there && j < n) wait(bar.k_full(ks), kp);
      if (!v_there && j > 0) wait(bar.v_full(vs), vp);
      k_there = v_there = false;
      const uint64_t kb = kd + (uint32_t)(ks * (C::kTile >> 4)), vb = vd + (uint32_t)(vs * (C::kTile >> 4));
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        if (t == 1 && !two) break;
        const uint32_t st = tmem + t * 128, ot = tmem + 256 + t * DP;
        if (t == 1) {  // while the first tile's MMAs run, and this one's weights are made
          const int k1 = ks + 1 == C::kStages ? 0 : ks + 1, v1 = j == 0 ? vs : vs + 1 == C::kStages ? 0 : vs + 1;
          k_there = j + 1 < n && mbar_test(bar.k_full(k1), k1 == 0 ? kp ^ 1 : kp);
          v_there = mbar_test(bar.v_full(v1), j > 0 && v1 == 0 ? vp ^ 1 : vp);
        }
        if (j > 0) {
          wait(bar.p_full(t), pp[t]);
          pp[t] ^= 1;
        }
        tc_fence_after();
        if (leader) {
          if (j > 0) {
#pragma unroll
            for (int i = 0; i < AT_KEYS / 16; ++i) mma_ts(ot, st + i * 8, vb + i * 128, io, j > 1 || i > 0);
            if (j == n) tc_commit(bar.o_full(t));
          }
          if (j < n) {
#pragma unroll
            for (int i = 0; i < DP / 16; ++i) {
              constexpr uint32_t block = C::kBlock >> 4;
              const uint32_t at = (i >> 2) * block + (i & 3) * 2;
              if (i * 16 < dims) mma_ss(st, qd + t * (C::kTile >> 4) + at, kb + at, is, i > 0);
            }
            tc_commit(bar.s_full(t));
          }
        }
        __syncwarp();
      }
      if (leader) {
        if (j > 0) tc_commit(bar.v_empty(vs));
        if (j < n) tc_commit(bar.k_empty(ks));
        if (j == n - 1) tc_commit(bar.q_empty());
      }
      if (!(ok = __all_sync(0xFFFFFFFFu, ok))) break;
      if (j > 0 && ++vs == C::kStages) {
        vs = 0;
        vp ^= 1;
      }
      if (j < n && ++ks == C::kStages) {
        ks = 0;
        kp ^= 1;
      }
    }
  }
  // nothing may be in flight when the CTA gives its memory back
  if (leader) tc_commit(bar.done());
  drain_wait(bar.done(), 0);
  __syncwarp();
}

// ---------------------------------------------------------------- softmax, output
// What is called out of line finds in shared memory: where the CTA's TMEM begins, and the maximum and sum of a row.
__device__ __forceinline__ uint32_t& tmem_base() {
  __shared__ uint32_t at;
  return at;
}
__device__ __forceinline__ float2& row_stats() {
  __shared__ float2 of[AT_BM];
  return of[threadIdx.x];
}

// What the loads took out of v where only some rows of the unit see it: weight times value, infinite or NaN, is added to the 32
// dims from d0 on of O, which hold the finite values already, for the keys [lo, hi) that a row sees. 256 tokens of one head of
// 128 dims, whose 255 keys of that kind hold nothing else, take 4 ms, far from the 200 that the other warps wait.
// Everything but the row's place comes out of memory and m, l and o are only written, so that the caller's loop over the
// steps has no registers to keep for this: with m handed over and O handed in, a prompt of 8192 tokens took 395 us for 387,
// one with a window of 1024 205 for 180.
template <typename T, int DP>
__device__ __noinline__ void add_odd(const AttnParams& p, const AttnUnit& u, int row, int lo, int hi, int d0, float& m, float& l,
                                     float (&o)[32]) {
  float sum[32];  // (o itself is the caller's, in memory)
  __syncwarp();
  tmem_ld32(tmem_base() + ((uint32_t)(threadIdx.x & 96) << 16) + 256 + (threadIdx.x >> 7) * DP + d0, sum);
  tmem_arrived(sum);
  m = row_stats().x;
  l = row_stats().y;
  const int tok = (int)p.group.div(u.row0 + row), g = u.row0 + row - tok * (int)p.group.d;
  const int64_t q_at = (int64_t)(u.seq.first + tok) * p.q_stride + (int64_t)(u.head * (int)p.group.d + g) * p.D;
  // keys that all rows of the unit see, as the loads have it
  const int all_lo = attn_range(p, u.seq, u.kv, (int)p.group.div(u.row0 + u.rows - 1)).x;
  const int all_hi = attn_range(p, u.seq, u.kv, (int)p.group.div(u.row0)).y;
  const int end = min(u.range.y, (u.range.x / AT_KEYS + u.s1) * AT_KEYS);
  const int lane = lane_id(), c16 = (lane & 15) * 8;
#pragma unroll 1
  for (int key = max(u.range.x, (u.range.x / AT_KEYS + u.s0) * AT_KEYS); key < end; ++key) {  // the same for all lanes
    if (key >= all_lo && key < all_hi) {
      key = all_hi - 1;
      continue;
    }
    const int j = (int)p.map.page.div(key), page = p.table[(int64_t)u.b * p.columns + j];
    if ((uint32_t)page >= (uint32_t)p.map.num_pages) continue;  // (reads as zeros)
    const int64_t off = page * p.map.page_stride + (int64_t)(key - j * (int)p.map.page.d) * p.map.token_stride +
                        (int64_t)u.head * p.map.head_stride;
    const T* v = static_cast<const T*>(p.v) + off + d0;
    const bool bad = lane < 4 && d0 + lane * 8 < p.D && any_nonfinite<T>(reinterpret_cast<const uint4*>(v)[lane & 3]);
    uint32_t pieces = __ballot_sync(0xFFFFFFFFu, bad);
    if (pieces == 0) continue;
    // the key's scores with the warp's rows: 16 lanes a row, a lane 8 dims
    float k8[8], s = 0.0f;
    unpack<T>(c16 < p.D ? *reinterpret_cast<const uint4*>(static_cast<const T*>(p.k) + off + c16) : make_uint4(0u, 0u, 0u, 0u), k8);
#pragma unroll 1
    for (int i0 = 0; i0 < 32; i0 += 8) {
      uint4 raw[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t at = __shfl_sync(0xFFFFFFFFu, q_at, i0 + 2 * i + (lane >> 4));
        raw[i] = *reinterpret_cast<const uint4*>(static_cast<const T*>(p.q) + at + (c16 < p.D ? c16 : 0));
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float q8[8], dot = 0.0f;
        unpack<T>(raw[i], q8);
#pragma unroll
        for (int e = 0; e < 8; ++e) dot = fmaf(q8[e], k8[e], dot);
        if (c16 >= p.D) dot = 0.0f;
#pragma unroll
        for (int d = 8; d; d >>= 1) dot += __shfl_xor_sync(0xFFFFFFFFu, dot, d);
        dot = __shfl_sync(0xFFFFFFFFu, dot, (lane & 1) * 16);  // of the first row to even lanes, of the second to odd ones
        if ((lane & ~1) == i0 + 2 * i) s = dot;
      }
    }
    if (key < lo || key >= hi) continue;
    const float w = exp2_fast(fmaf(s, p.scale_log2, -weight_base<T>(m, p.scale_log2)));
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      if ((pieces >> c & 1) == 0) continue;
      float x[8];
      unpack<T>(reinterpret_cast<const uint4*>(v)[c], x);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (!isfinite(x[e])) sum[c * 8 + e] = fmaf(w, x[e], sum[c * 8 + e]);
    }
  }
#pragma unroll
  for (int i = 0; i < 32; ++i) o[i] = sum[i];
}

// Of 32 scores of a row.
template <bool EDGE>
__device__ __forceinline__ void hide(float (&s)[32], int from, int to) {  // all but columns [from, to)
  if constexpr (EDGE) {
#pragma unroll
    for (int c = 0; c < 32; ++c)
      if (c < from || c >= to) s[c] = -INFINITY;
  }
}
__device__ __forceinline__ float greatest(const float (&s)[32], float top) {
  float x[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
  for (int c = 4; c < 28; c += 8)
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = max3(x[i], s[c + 2 * i], s[c + 2 * i + 1]);
  return max3(max3(top, max3(x[0], x[1], s[28]), max3(x[2], x[3], s[29])), s[30], s[31]);
}
template <typename T>
__device__ __forceinline__ void weights(const float (&s)[32], uint32_t* w, float (&sum)[4], float scale, float mb) {
#pragma unroll
  for (int c = 0; c < 16; ++c) {
    float u, v;
    fma2(u, v, s[2 * c], s[2 * c + 1], scale, -mb);
    u = exp2_fast(u);
    v = exp2_fast(v);
    add2(sum[2 * (c & 1)], sum[2 * (c & 1) + 1], u, v);
    w[c] = pack2<T>(u, v);  // half a step of the cache's type, against a result of that type
  }
}
// One step of a row: S (128 columns, of which the row sees [from, to)) into P, m and l brought up to date, O rescaled.
template <typename T, bool EDGE>
__device__ __forceinline__ void softmax_step(uint32_t st, uint32_t ot, int dims, bool first, int from, int to, float scale, float& m,
                                             float& l) {
  float a[2][32], b[2][32];
  uint32_t w[2][32];
  float top, sum[4];
  if (first) {  // no maximum yet
    top = -INFINITY;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      tmem_ld32(st + i * 32, a[0]);
      tmem_arrived(a[0]);
      hide<EDGE>(a[0], from - i * 32, to - i * 32);
      top = greatest(a[0], top);
    }
    m = top;
  }
  // The weights under the maximum so far, and the step's maximum beside them; again if it had grown too much.
  for (;;) {
    const float mb = weight_base<T>(m, scale);
    top = m;
    sum[0] = sum[1] = sum[2] = sum[3] = 0.0f;
    tmem_ld32(st, a[0]);
    tmem_ld32(st + 32, a[1]);
    tmem_arrived(a[0]);
    tmem_arrived(a[1]);
    tmem_ld32(st + 64, b[0]);
    tmem_ld32(st + 96, b[1]);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      hide<EDGE>(a[i], from - i * 32, to - i * 32);
      top = greatest(a[i], top);
      weights<T>(a[i], w[0] + 16 * i, sum, scale, mb);
    }
    tmem_arrived(b[0]);
    tmem_arrived(b[1]);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      hide<EDGE>(b[i], from - 64 - i * 32, to - 64 - i * 32);
      top = greatest(b[i], top);
      weights<T>(b[i], w[1] + 16 * i, sum, scale, mb);
    }
    if (!__any_sync(0xFFFFFFFFu, (top - safe_max(m)) * scale > AT_GROWTH || (m == -INFINITY && top > m))) break;
    const float f = exp2_fast((m - safe_max(top)) * scale);
    m = top;
    l *= f;
    if (!first) {
#pragma unroll 1
      for (int d = 0; d < dims; d += 8) tmem_scale8(ot + d, f);
    }
  }
  l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
  tmem_st32(st, w[0]);
  tmem_st32(st + 32, w[1]);
  tmem_st_wait();
  tc_fence_before();
}

template <typename T, int DP>
__device__ __forceinline__ void softmax_role(const AttnParams& p, const AttnRun& run, const TileBars<DP>& bar, uint32_t tmem,
                                             volatile int* odd, volatile uint32_t* arrived, uint8_t* stage) {
  const int t = threadIdx.x >> 7, row = threadIdx.x & 127;
  const uint32_t lanes = (uint32_t)(row & 96) << 16;  // this warp's 32 lanes of TMEM
  const uint32_t st = tmem + lanes + t * 128, ot = tmem + lanes + 256 + t * DP;
  const int dims = (p.D + 15) / 16 * 16;
  int units = 0;
  uint32_t sp = 0, op = 0, jp = 0;
  bool ok = true;
  AttnWalk walk(run);
  for (AttnUnit u; ok && walk.next<AT_BM, AT_KEYS, AT_OH>(p, run, u); ++units) {
    if (t * 128 >= u.rows) continue;  // (as the MMAs leave the tile out)
    const int last = min(u.rows, t * 128 + 128) - 1, r = min(t * 128 + row, last);
    const bool real = t * 128 + row <= last, idle = t * 128 + (row & 96) > last;  // idle: a warp without rows
    const int2 see = attn_range(p, u.seq, u.kv, (int)p.group.div(u.row0 + r));
    const int all_lo = attn_range(p, u.seq, u.kv, (int)p.group.div(u.row0 + last)).x;
    const int all_hi = attn_range(p, u.seq, u.kv, (int)p.group.div(u.row0 + t * 128)).y;
    float m = -INFINITY, l = 0.0f;
    const int k00 = (u.range.x / AT_KEYS + u.s0) * AT_KEYS, n = u.s1 - u.s0;
    // steps [in0, in1) are all visible to all rows
    const int in0 = all_lo > k00 ? (all_lo - k00 + AT_KEYS - 1) / AT_KEYS : 0, in1 = all_hi > k00 ? (all_hi - k00) / AT_KEYS : 0;
    for (int j = 0; j < n; ++j) {
      if (!(ok = warp_wait(bar.s_full(t), sp, p.err))) break;
      sp ^= 1;
      tc_fence_after();
      if (idle) {  // (what P holds of rows that there are not reaches only rows of O that there are not)
      } else if (j >= in0 && j < in1)
        softmax_step<T, false>(st, ot, dims, j == 0, 0, 0, p.scale_log2, m, l);
      else
        softmax_step<T, true>(st, ot, dims, j == 0, see.x - k00 - j * AT_KEYS, see.y - k00 - j * AT_KEYS, p.scale_log2, m, l);
      __syncwarp();
      if (lane_id() == 0) mbar_arrive(bar.p_full(t));
    }
    if (!ok || !(ok = warp_wait(bar.o_full(t), op, p.err))) break;
    op ^= 1;
    tc_fence_after();
    if (!idle && odd[units % AT_ODD] == units + 1) {
      const int k0 = (u.range.x / AT_KEYS + u.s0) * AT_KEYS, k1 = (u.range.x / AT_KEYS + u.s1) * AT_KEYS;
      row_stats() = make_float2(m, l);
      for (int d = 0; d < dims; d += 32) {
        float o[32];
        uint32_t w[32];
        add_odd<T, DP>(p, u, r, max(see.x, k0), min(see.y, k1), d, m, l, o);
#pragma unroll
        for (int c = 0; c < 32; ++c) w[c] = __float_as_uint(o[c]);
        __syncwarp();
        tmem_st32(ot + d, w);
      }
      tmem_st_wait();
    }
    const int tok = (int)p.group.div(u.row0 + r), g = u.row0 + r - tok * (int)p.group.d;
    const int64_t tq = u.seq.first + tok;
    const int hq = u.head * (int)p.group.d + g;
    const int64_t at = real ? tq * p.out_stride + (int64_t)hq * p.D : -1;
    const bool none = see.x >= see.y;  // a row without keys is 0 (its sums are); one whose scores are all -infinity is 0 / 0
    // 32 dims of the warp's rows, through shared memory: four lanes write a row's 64 bytes
    auto finish = [&](float (&o)[32], int d, float inv) {
      const int lane = row & 31;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = o[c * 8 + e] * inv;
        *reinterpret_cast<uint4*>(stage + lane * 64 + ((c ^ ((lane >> 1) & 3)) << 4)) = pack<T>(v);
      }
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int rr = i * 8 + (lane >> 2), c = lane & 3;
        const int64_t to = __shfl_sync(0xFFFFFFFFu, at, rr);
        if (to >= 0 && d + c * 8 < p.D)
          *reinterpret_cast<uint4*>(static_cast<T*>(p.out) + to + d + c * 8) =
              *reinterpret_cast<const uint4*>(stage + rr * 64 + ((c ^ ((rr >> 1) & 3)) << 4));
      }
      __syncwarp();
    };
    auto finish_lse = [&](float M, float sum) {
      if (real && p.lse != nullptr) p.lse[tq * p.q_heads + hq] = none ? -INFINITY : weights_lse<T>(M, p.scale, sum);
    };
    if (u.s0 == 0 && u.s1 == u.n) {
      const float inv = none ? 0.0f : __fdiv_rn(1.0f, l);
#pragma unroll 1
      for (int d = 0; d < dims && !idle; d += 32) {
        float o[32];
        tmem_ld32(ot + d, o);
        tmem_arrived(o);
        finish(o, d, inv);
      }
      finish_lse(m, l);
    } else {
      const int c0 = attn_owner(run, u.first), c1 = attn_owner(run, u.first + u.n - 1);
      float2* stats = reinterpret_cast<float2*>(p.ws + kAttnStats);
      float* sums = reinterpret_cast<float*>(p.ws + kAttnSums);
      const int lane = row & 31, rows_t = last + 1 - t * 128;
      auto slot = [&](int c) { return (int64_t)(2 * c + (c == c0 ? 1 : 0)) * AT_BM + t * 128; };  // of CTA c: this tile's rows
      // Few rows lie one after the other, a warp's lanes across them; of many, vectors of four dims of all rows lie side by
      // side, a lane a row.
      const bool few = rows_t <= AT_FEW;
      auto vec = [&](int64_t s, int d) { return reinterpret_cast<float4*>(sums + s * DP) + (d / 4) * 128 + row; };
      const int64_t mine = slot(blockIdx.x);
      auto meet = [&] {  // the tile's four warps
        __syncwarp();
        if (lane == 0) mbar_arrive(bar.join(t));
        ok = warp_wait(bar.join(t), jp, p.err);
        jp ^= 1;
        return ok;
      };
      uint32_t* count = reinterpret_cast<uint32_t*>(p.ws + kAttnCounters) + 2 * c0 + t;
      const uint32_t others = (uint32_t)(c1 - c0);
      // Where all others have left their parts, this one's need not be written: it is added out of TMEM, in its turn.
      if (row == 0) {
        arrived[t] = *(volatile uint32_t*)count;
        __threadfence();
      }
      if (!meet()) break;
      bool last_one = arrived[t] == others;
      const bool kept = last_one && !few;
      if (!kept) {
        if (!idle) {
          __stcg(stats + mine + row, make_float2(m, l));
#pragma unroll 1
          for (int d = 0; d < dims; d += 32) {  // few: through shared memory, 16 dims at a time, four lanes to a row's 64 bytes
            float o[32];
            tmem_ld32(ot + d, o);
            tmem_arrived(o);
            if (!few) {
#pragma unroll
              for (int c = 0; c < 32; c += 4) __stcg(vec(mine, d + c), make_float4(o[c], o[c + 1], o[c + 2], o[c + 3]));
              continue;
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
              for (int c = 0; c < 4; ++c)
                *reinterpret_cast<float4*>(stage + lane * 64 + ((c ^ ((lane >> 1) & 3)) << 4)) =
                    make_float4(o[h * 16 + c * 4], o[h * 16 + c * 4 + 1], o[h * 16 + c * 4 + 2], o[h * 16 + c * 4 + 3]);
              __syncwarp();
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int rr = i * 8 + (lane >> 2), c = lane & 3;
                __stcg(reinterpret_cast<float4*>(sums + (mine + (row & 96) + rr) * DP + d + h * 16 + c * 4),
                       *reinterpret_cast<const float4*>(stage + rr * 64 + ((c ^ ((rr >> 1) & 3)) << 4)));
              }
              __syncwarp();
            }
          }
        }
        if (!meet()) break;
        if (!last_one) {
          if (row == 0) {  // its fences stand for the tile's writes before this, and for its reads after the next meeting
            __threadfence();
            arrived[t] = atomicAdd(count, 1u);
            __threadfence();
          }
          if (!meet()) break;
          last_one = arrived[t] == others;
        }
      }
      if (last_one) {  // adds all parts in order
        if (row == 0) *count = 0;
        // Few: a warp takes four rows at a time, eight lanes a row; a lane four dims of every 32, and the weight of every eighth
        // part.
        const int sub = lane & 7;
        for (int r0 = (row >> 5) * 4; few && r0 < rows_t; r0 += 16) {
          const int rr = min(r0 + (lane >> 3), rows_t - 1);
          float M = -INFINITY, sum = 0.0f;
          for (int c = c0 + sub; c <= c1; c += 8) M = fmaxf(M, __ldcg(stats + slot(c) + rr).x);
#pragma unroll
          for (int d = 4; d; d >>= 1) M = fmaxf(M, __shfl_xor_sync(0xFFFFFFFFu, M, d));
          constexpr int NV = DP / 32;
          float4 o[NV];
#pragma unroll
          for (int d = 0; d < NV; ++d) o[d] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          for (int cb = c0; cb <= c1; cb += 8) {
            const int n = min(8, c1 + 1 - cb);
            float f = 0.0f, w = 0.0f;
            if (sub < n) {
              const float2 ml = __ldcg(stats + slot(cb + sub) + rr);
              f = exp2_fast((ml.x - safe_max(M)) * p.scale_log2);
              w = ml.y * f;
            }
#pragma unroll
            for (int d = 4; d; d >>= 1) w += __shfl_xor_sync(0xFFFFFFFFu, w, d);
            sum += w;
#pragma unroll 4
            for (int c = 0; c < n; ++c) {
              const float fc = __shfl_sync(0xFFFFFFFFu, f, (lane & 24) + c);
              const float4* part = reinterpret_cast<const float4*>(sums + (slot(cb + c) + rr) * DP) + sub;
#pragma unroll
              for (int d = 0; d < NV; ++d) {
                if (d * 32 < dims) {
                  const float4 v = __ldcg(part + d * 8);
                  o[d].x = fmaf(v.x, fc, o[d].x);
                  o[d].y = fmaf(v.y, fc, o[d].y);
                  o[d].z = fmaf(v.z, fc, o[d].z);
                  o[d].w = fmaf(v.w, fc, o[d].w);
                }
              }
            }
          }
          if (r0 + (lane >> 3) < rows_t) {
            const int gr = u.row0 + t * 128 + rr, rtok = (int)p.group.div(gr), rhq = u.head * (int)p.group.d + gr - rtok * (int)p.group.d;
            const int2 sees = attn_range(p, u.seq, u.kv, rtok);
            const bool nothing = sees.x >= sees.y;
            const float inv = nothing ? 0.0f : __fdiv_rn(1.0f, sum);
            const int64_t rt = u.seq.first + rtok;
            T* to = static_cast<T*>(p.out) + rt * p.out_stride + (int64_t)rhq * p.D;
#pragma unroll
            for (int d = 0; d < NV; ++d)
              if (d * 32 + sub * 4 < p.D)
                *reinterpret_cast<uint2*>(to + d * 32 + sub * 4) =
                    make_uint2(pack2<T>(o[d].x * inv, o[d].y * inv), pack2<T>(o[d].z * inv, o[d].w * inv));
            if (sub == 0 && p.lse != nullptr) p.lse[rt * p.q_heads + rhq] = nothing ? -INFINITY : weights_lse<T>(M, p.scale, sum);
          }
        }
        if (!few && !idle) {
          auto stat = [&](int c) { return c == (int)blockIdx.x ? make_float2(m, l) : __ldcg(stats + slot(c) + row); };
          float M = -INFINITY, sum = 0.0f;
#pragma unroll 1
          for (int c = c0; c <= c1; ++c) {
            const float2 ml = stat(c);
            const float nm = fmaxf(M, ml.x);
            sum = fmaf(sum, exp2_fast((M - safe_max(nm)) * p.scale_log2), ml.y * exp2_fast((ml.x - safe_max(nm)) * p.scale_log2));
            M = nm;
          }
          const float inv = none ? 0.0f : __fdiv_rn(1.0f, sum);
#pragma unroll 1
          for (int d = 0; d < dims; d += 32) {
            float o[32], own[32];
            tmem_ld32(ot + d, own);
#pragma unroll
            for (int c = 0; c < 32; ++c) o[c] = 0.0f;
            tmem_arrived(own);
#pragma unroll 1
            for (int c = c0; c <= c1; ++c) {
              const float f = exp2_fast((stat(c).x - safe_max(M)) * p.scale_log2);
              if (c == (int)blockIdx.x) {
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = fmaf(own[e], f, o[e]);
                continue;
              }
              float4 v[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) v[e] = __ldcg(vec(slot(c), d + 4 * e));
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                o[4 * e] = fmaf(v[e].x, f, o[4 * e]);
                o[4 * e + 1] = fmaf(v[e].y, f, o[4 * e + 1]);
                o[4 * e + 2] = fmaf(v[e].z, f, o[4 * e + 2]);
                o[4 * e + 3] = fmaf(v[e].w, f, o[4 * e + 3]);
              }
            }
            finish(o, d, inv);
          }
          finish_lse(M, sum);
        }
      }
      __syncwarp();
    }
    tc_fence_before();  // O has been read: the next unit's first P V, which waits for this group's P, may overwrite it
  }
}

template <typename T, int DP, int MODE>
__global__ void __launch_bounds__(AT_THREADS, 1) attn_tile_kernel(AttnParams p, const __grid_constant__ TileMaps maps) {
  using C = TileCfg<DP>;
  extern __shared__ uint8_t raw[];
  __shared__ uint32_t arrived[2], skip;
  uint32_t& tmem_at = tmem_base();
  __shared__ int odd[AT_ODD];  // [unit % AT_ODD]: unit + 1 if a v that only some of its rows see is not finite
  uint8_t* sm = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
  const uint32_t sm32 = smem_u32(sm);
  const TileBars<DP> bar{sm32 + C::kBars};
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(bar.k_full(s), 1);
      mbar_init(bar.v_full(s), 1);
      mbar_init(bar.k_empty(s), 1);
      mbar_init(bar.v_empty(s), 1);
    }
    mbar_init(bar.q_full(), maps.q_box ? 1 : 2);  // both loading warps bring a tile without boxes
    mbar_init(bar.q_empty(), 1);
    for (int t = 0; t < 2; ++t) {
      mbar_init(bar.s_full(t), 1);
      mbar_init(bar.p_full(t), 4);
      mbar_init(bar.o_full(t), 1);
      mbar_init(bar.join(t), 4);
    }
    mbar_init(bar.done(), 1);
    mbar_init(bar.landed(), 1);
    fence_mbar_init();
    for (int i = 0; i < AT_ODD; ++i) odd[i] = 0;
  }
  if (threadIdx.x == 32) {
    for (const CUtensorMap* m : {&maps.k, &maps.v, &maps.q})
      asm volatile("prefetch.tensormap [%0];" ::"l"((uint64_t)m) : "memory");
  }
  if (warp == 8) {
    tmem_alloc(smem_u32(&tmem_at), 512);
    tmem_relinquish();
  }
  pdl_wait();
  pdl_trigger();
  if (threadIdx.x == 0) skip = *(volatile uint32_t*)p.err & kAbortMask;
  AttnRun run = attn_plan<AT_BM, AT_KEYS, AT_OH, AT_MIN, AT_THREADS>(p, reinterpret_cast<int64_t*>(sm));
  fence_proxy_async_smem();  // the division's sums lie where loads will
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (skip) run.end = run.begin;  // an earlier call gave up
  const uint32_t tmem = tmem_at;
  if (warp < 8) {
    softmax_role<T, DP>(p, run, bar, tmem, odd, arrived, sm + C::kOut + warp * 2048);
  } else if (warp == 8) {
    mma_role<T, DP>(p, run, bar, sm32, tmem);
  } else if (warp == 9) {
    load_role<T, DP, MODE, 0>(p, maps, run, bar, sm, sm32, odd);
  } else {
    load_role<T, DP, MODE, 1>(p, maps, run, bar, sm, sm32, odd);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 8) tmem_dealloc(tmem, 512);
}

template <typename T, int DP, int MODE>
fp4moe_status attn_tile_run(const AttnParams& p, const TileMaps& maps, int nsm, cudaStream_t st) {
  using C = TileCfg<DP>;
  static PerDevice done;
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return FP4MOE_CUDA_ERROR;
  if (done.get(dev, [] {
        return cudaFuncSetAttribute(attn_tile_kernel<T, DP, MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem) ==
                       cudaSuccess
                   ? 1
                   : 0;
      }) <= 0)
    return FP4MOE_CUDA_ERROR;
  return launch_pdl(attn_tile_kernel<T, DP, MODE>, dim3((unsigned)nsm), dim3(AT_THREADS), C::kSmem, st, p, maps) == cudaSuccess
             ? FP4MOE_OK
             : FP4MOE_CUDA_ERROR;
}

decltype(&cuTensorMapEncodeTiled) tiled_encoder() {
  static const auto fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<decltype(&cuTensorMapEncodeTiled)>(f);
  }();
  return fn;
}
// dims and box from the innermost on; strides of the others in elements of 2 bytes, that of a dimension of one element
// being of no account. False where a map cannot say it.
bool encode_boxes(CUtensorMap* m, int32_t dtype, const void* base, int rank, const int64_t* dims, const int64_t* strides,
                  const uint32_t* box) {
  const auto encode = tiled_encoder();
  if (encode == nullptr) return false;
  cuuint64_t d[4], s[3];
  cuuint32_t b[4], es[4] = {1, 1, 1, 1};
  for (int i = 0; i < rank; ++i) {
    d[i] = (cuuint64_t)dims[i];
    b[i] = box[i];
    if (i == 0) continue;
    s[i - 1] = dims[i] == 1 ? 16 : (cuuint64_t)strides[i - 1] * 2;
    if (s[i - 1] == 0 || s[i - 1] >= (1ull << 40)) return false;
  }
  return encode(m, dtype == FP4MOE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, (cuuint32_t)rank,
                const_cast<void*>(base), d, s, b, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, int DP>
fp4moe_status attn_tile_mode(const AttnParams& p, const TileMaps& maps, int nsm, cudaStream_t st) {
  return maps.rows > 1    ? attn_tile_run<T, DP, kBoxes>(p, maps, nsm, st)
         : maps.rows == 1 ? attn_tile_run<T, DP, kGathers>(p, maps, nsm, st)
                          : attn_tile_run<T, DP, kCopies>(p, maps, nsm, st);
}
template <typename T>
fp4moe_status attn_tile_typed(const AttnParams& p, const TileMaps& maps, int nsm, cudaStream_t st) {
  return p.D <= 64 ? attn_tile_mode<T, 64>(p, maps, nsm, st) : attn_tile_mode<T, 128>(p, maps, nsm, st);
}

}  // namespace

fp4moe_status attn_tile_launch(int32_t dtype, const AttnParams& p, int nsm, cudaStream_t st) {
  TileMaps maps{};
  int rows = 128;  // whole 8-row swizzle atoms that divide a page
  while (p.map.page.d % rows != 0) rows /= 2;
  const int64_t kd[4] = {p.D, p.kv_heads, p.map.page.d, p.map.num_pages};
  const int64_t ks[3] = {p.map.head_stride, p.map.token_stride, p.map.page_stride};
  const uint32_t kb[4] = {64, 1, (uint32_t)rows, 1};
  if (rows >= 8 && encode_boxes(&maps.k, dtype, p.k, 4, kd, ks, kb) && encode_boxes(&maps.v, dtype, p.v, 4, kd, ks, kb))
    maps.rows = rows;
  // A token's heads as one row, where the slots lie evenly and an MMA step's dims are all of one head: what lies behind a
  // head is brought with it, and 0 (q's) times that may be NaN.
  if (maps.rows == 0 && p.D % 16 == 0) {
    const int64_t slots = (int64_t)p.map.num_pages * p.map.page.d, width = (p.kv_heads - 1) * p.map.head_stride + p.D;
    const int64_t apart = p.map.page.d == 1 ? p.map.page_stride : p.map.token_stride;
    const bool even = p.map.page.d == 1 || p.map.num_pages == 1 || p.map.page_stride == p.map.page.d * p.map.token_stride;
    const int64_t gd[2] = {width, slots}, gs[1] = {apart};
    const uint32_t gb[2] = {64, 1};
    if (even && width <= INT32_MAX && encode_boxes(&maps.k, dtype, p.k, 2, gd, gs, gb) &&
        encode_boxes(&maps.v, dtype, p.v, 2, gd, gs, gb))
      maps.rows = 1;
  }
  if (128 % p.group.d == 0) {
    const int64_t qd[3] = {p.D, p.q_heads, p.T}, qs[2] = {p.D, p.q_stride};
    const uint32_t qb[3] = {64, p.group.d, 128 / p.group.d};
    maps.q_box = encode_boxes(&maps.q, dtype, p.q, 3, qd, qs, qb);
  }
  return dtype == FP4MOE_BF16 ? attn_tile_typed<__nv_bfloat16>(p, maps, nsm, st) : attn_tile_typed<__half>(p, maps, nsm, st);
}

}  // namespace fp4moe
