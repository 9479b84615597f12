// What both attention kernels share (attn.cu, attntile.cu): the division of the work, the rows of a tile, and the join of
// what several CTAs make of one tile.
//
// Rows. The rows of a sequence and kv head are its (token, query head of the group) pairs, token by token: they read the
// same keys. A tile is BM of them. It sees the keys [lo, hi), and costs ceil(hi / S) - floor(lo / S) slices of S keys (at
// least one: a tile without keys still has to be written).
//
// Division. A tile and kv head costs OH (to begin and end it) and one for each slice. The costs of all of them, in order,
// are cut into gridDim.x equal runs, one for each CTA, whatever the lengths are: a long sequence is spread over many
// CTAs, and many short ones are shared out evenly. A CTA's run holds parts of at most two tiles that other CTAs share:
// the one that it starts in (begun by an earlier CTA) and the one that it ends in. Each CTA finds its run by itself from
// q_offset and kv_len.
//
// Join. A CTA leaves the unnormalised sums of its part (fp32, under its own maximum) in the workspace and counts itself
// in; the last one adds the parts in the order of the CTAs, so equal inputs give equal bits, and sets the count back.
#pragma once

#include "paged.cuh"

namespace fp4moe {

constexpr int kAttnMaxCtas = 240;
constexpr int kAttnTileRows = 256;  // of the larger kernel
constexpr size_t kAttnCounters = 256;  // byte offset of the counters, two a CTA, zero between calls
constexpr size_t kAttnStats = 4096;    // [2 a CTA][rows] {maximum, sum}
constexpr size_t kAttnSums = kAttnStats + (size_t)2 * kAttnMaxCtas * kAttnTileRows * 8;  // [2 a CTA][rows][dims] fp32
static_assert(kAttnCounters + 8 * kAttnMaxCtas <= kAttnStats, "counters fit");
static_assert(kAttnSums + (size_t)2 * kAttnMaxCtas * kAttnTileRows * 128 * 4 <= FP4MOE_ATTENTION_WORKSPACE_BYTES,
              "workspace");

struct AttnParams {
  CacheMap map;
  const void *k, *v, *q;
  void* out;
  float* lse;
  const int32_t *table, *kv_len, *q_offset;
  int64_t q_stride, out_stride;
  int B, T, q_heads, kv_heads, D, columns;
  FastDiv group;  // query heads of a kv head
  int causal, window;
  float scale, scale_log2;
  uint8_t* ws;
  uint32_t* err;
};

// A sequence: its first row, number of rows (of one kv head) and keys.
struct AttnSeq {
  int first, rows, keys, tokens;
};
__device__ __forceinline__ AttnSeq attn_seq(const AttnParams& p, int q0, int q1, int kv) {
  AttnSeq s;
  q0 = max(0, min(q0, p.T));
  q1 = max(q0, min(q1, p.T));
  s.first = q0;
  s.tokens = q1 - q0;
  s.rows = s.tokens * (int)p.group.d;
  const int64_t room = (int64_t)p.columns * p.map.page.d;
  s.keys = kv < 0 ? 0 : (int64_t)kv > room ? (int)room : kv;
  return s;
}
// Keys that token i of a sequence sees: [lo, hi).
__device__ __forceinline__ int2 attn_range(const AttnParams& p, const AttnSeq& s, int kv, int i) {
  // the last row's position is kv - 1; keys past the table's columns are missing
  const int64_t pos = (int64_t)kv - s.tokens + i;
  int64_t hi = p.causal ? pos + 1 : (int64_t)s.keys;
  int64_t lo = p.window ? pos + 1 - p.window : 0;
  hi = hi < 0 ? 0 : hi > s.keys ? s.keys : hi;
  lo = lo < 0 ? 0 : lo > hi ? hi : lo;
  return make_int2((int)lo, (int)hi);
}
// Tiles of a sequence. (rows may be 2^31 - 1: no sum here passes it)
template <int BM>
__device__ __forceinline__ int attn_tiles(int rows) {
  return rows / BM + (rows % BM != 0);
}
// Keys that any row of tile `i` sees; a superset with the same ends.
template <int BM>
__device__ __forceinline__ int2 attn_tile_range(const AttnParams& p, const AttnSeq& s, int kv, int i) {
  const int r0 = i * BM, r1 = r0 + min(BM, s.rows - r0) - 1;
  const int lo = attn_range(p, s, kv, (int)p.group.div(r0)).x, hi = attn_range(p, s, kv, (int)p.group.div(r1)).y;
  return make_int2(min(lo, hi), hi);
}
template <int S>
__device__ __forceinline__ int attn_slices(int2 r) {
  return max(1, (r.y + S - 1) / S - r.x / S);
}

// Where a CTA's run of costs lies, and where it starts.
struct AttnRun {
  int64_t total, begin, end;  // of the call, and the CTA's own
  int ctas;                   // CTAs that have a run, of a cost of MIN at least where there is that much
  int64_t each;               // total / ctas,
  int rest;                   // and what that leaves
  int seq, tile, head;        // of `begin`
  int at;                     // its place in its tile and head: the first OH are before slice 0
};

// Where the run of a CTA begins: total * cta / ctas.
__device__ __forceinline__ int64_t attn_begin(const AttnRun& r, int cta) {
  return r.each * cta + (uint32_t)(r.rest * cta) / (uint32_t)r.ctas;
}
// The CTA whose run holds x: about where x / total is, then exactly.
__device__ __forceinline__ int attn_owner(const AttnRun& r, int64_t x) {
  int c = min((int)((float)x / (float)r.total * (float)r.ctas), r.ctas - 1);
  while (c + 1 < r.ctas && attn_begin(r, c + 1) <= x) ++c;
  while (c > 0 && attn_begin(r, c) > x) --c;
  return c;
}

// a / b of non-negative values, which mostly fit 32 bits.
__device__ __forceinline__ int64_t attn_div(int64_t a, int64_t b) {
  return ((uint64_t)(a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}

// Cost of sequence b, by all lanes of a warp, each with a sequence of its own (or none: b >= B); short sequences by their
// lane, those of several tiles by the warp. bad: whether a length is out of range.
template <int BM, int S, int OH>
__device__ __forceinline__ int64_t attn_cost(const AttnParams& p, int b, uint32_t& bad) {
  const int lane = lane_id();
  int64_t w = 0;
  int big = 0, kv = 0;
  AttnSeq s{};
  if (b < p.B) {
    const int q0 = p.q_offset[b], q1 = p.q_offset[b + 1];
    kv = p.kv_len[b];
    s = attn_seq(p, q0, q1, kv);
    if (s.keys != kv && s.rows > 0) bad = 1;
    if (s.rows > BM) big = 1;
    else if (s.rows > 0) w = (int64_t)(OH + attn_slices<S>(attn_tile_range<BM>(p, s, kv, 0))) * p.kv_heads;
  }
  for (uint32_t m = __ballot_sync(0xFFFFFFFFu, big); m; m &= m - 1) {
    const int src = __ffs(m) - 1;
    AttnSeq o;
    o.first = __shfl_sync(0xFFFFFFFFu, s.first, src);
    o.rows = __shfl_sync(0xFFFFFFFFu, s.rows, src);
    o.keys = __shfl_sync(0xFFFFFFFFu, s.keys, src);
    o.tokens = __shfl_sync(0xFFFFFFFFu, s.tokens, src);
    const int okv = __shfl_sync(0xFFFFFFFFu, kv, src);
    int64_t sum = 0;
    for (int t = lane; t < attn_tiles<BM>(o.rows); t += 32) sum += OH + attn_slices<S>(attn_tile_range<BM>(p, o, okv, t));
#pragma unroll
    for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
    if (lane == src) w = sum * p.kv_heads;
  }
  return w;
}
__device__ __forceinline__ int64_t attn_warp_sum(int64_t x) {  // inclusive
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xFFFFFFFFu, x, o);
    if ((int)lane_id() >= o) x += y;
  }
  return x;
}

// All threads of the CTA call this. sums: (B + THREADS / 32 + 2) * 8 bytes of shared memory, free again afterwards.
template <int BM, int S, int OH, int MIN, int THREADS>
__device__ __forceinline__ AttnRun attn_plan(const AttnParams& p, int64_t* sums) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int WARPS = THREADS / 32;
  int64_t* part = sums;              // [WARPS + 1]
  int64_t* upto = sums + WARPS + 1;  // [B] costs of the sequences up to and with b
  uint32_t bad = 0;
  const bool few = p.B <= 32;  // every warp for itself: no shared memory, and no barrier but the last
  int64_t before = 0, total = 0, mine = 0;
  if (few) {
    mine = attn_warp_sum(attn_cost<BM, S, OH>(p, lane, bad));
    total = __shfl_sync(0xFFFFFFFFu, mine, 31);
  } else {
    const int per = (p.B + THREADS - 1) / THREADS;
    for (int i = 0; i < per; ++i) {
      const int b = i * THREADS + tid;
      const int64_t w = attn_cost<BM, S, OH>(p, b, bad);
      if (b < p.B) upto[b] = w;
    }
    __syncthreads();
    // running sum: a thread's stretch of sequences, then the threads
    const int b0 = min(tid * per, p.B), b1 = min(b0 + per, p.B);
    for (int b = b0; b < b1; ++b) mine += upto[b];
    const int64_t x = attn_warp_sum(mine);
    if (lane == 31) part[warp] = x;
    __syncthreads();
    before = x - mine;
    for (int w = 0; w < WARPS; ++w) {
      if (w < warp) before += part[w];
      total += part[w];
    }
    for (int b = b0; b < b1; ++b) {
      before += upto[b];
      upto[b] = before;
    }
    __syncthreads();
  }
  if (bad) raise_error(p.err, FP4MOE_ERR_PAGE);
  AttnRun r;
  r.total = total;
  r.ctas = (int)max((int64_t)1, min(attn_div(total, MIN), (int64_t)gridDim.x));
  r.each = attn_div(total, r.ctas);
  r.rest = (int)(total - r.each * r.ctas);
  r.begin = (int)blockIdx.x < r.ctas ? attn_begin(r, blockIdx.x) : 0;
  r.end = (int)blockIdx.x < r.ctas ? attn_begin(r, blockIdx.x + 1) : 0;
  r.seq = r.tile = r.head = r.at = 0;
  if (r.begin < r.end) {
    int64_t left;
    if (few) {
      r.seq = __ffs(__ballot_sync(0xFFFFFFFFu, mine > r.begin)) - 1;
      const int64_t y = __shfl_sync(0xFFFFFFFFu, mine, max(r.seq - 1, 0));
      left = r.begin - (r.seq ? y : 0);
    } else {
      int lo = 0, hi = p.B - 1;  // first sequence with upto > begin
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (upto[mid] > r.begin) hi = mid;
        else lo = mid + 1;
      }
      r.seq = lo;
      left = r.begin - (lo ? upto[lo - 1] : 0);
    }
    const int kv = p.kv_len[r.seq];
    const AttnSeq s = attn_seq(p, p.q_offset[r.seq], p.q_offset[r.seq + 1], kv);
    const int tiles = attn_tiles<BM>(s.rows);
    for (int t0 = 0; t0 < tiles; t0 += 32) {  // every warp for itself
      const int t = t0 + lane;
      const int n = t < tiles ? OH + attn_slices<S>(attn_tile_range<BM>(p, s, kv, t)) : 0;
      const int64_t w = (int64_t)n * p.kv_heads, y = attn_warp_sum(w);
      const uint32_t hit = __ballot_sync(0xFFFFFFFFu, t < tiles && y > left);
      if (hit) {
        const int src = __ffs(hit) - 1;
        r.tile = t0 + src;
        left -= __shfl_sync(0xFFFFFFFFu, y - w, src);
        const int cost = __shfl_sync(0xFFFFFFFFu, n, src);
        r.head = (int)attn_div(left, cost);
        r.at = (int)(left - (int64_t)r.head * cost);
        break;
      }
      left -= __shfl_sync(0xFFFFFFFFu, y, 31);
    }
  }
  __syncthreads();
  return r;
}

// What a CTA does in one go: slices [s0, s1) of one tile and kv head.
struct AttnUnit {
  AttnSeq seq;
  int kv, b, tile, head;
  int row0, rows;  // the tile's first row of the sequence, and its rows
  int2 range;      // keys that any of them sees
  int n, s0, s1;   // slices of the tile, and those of this unit
  int64_t first;   // slice 0's place among the call's costs
};
// The units of a run, one after the other.
struct AttnWalk {
  int64_t x;
  int b, tile, head, at;
  int read = -1, kv = 0;  // the sequence that `seq` is
  AttnSeq seq{};
  __device__ __forceinline__ explicit AttnWalk(const AttnRun& r)
      : x(r.begin), b(r.seq), tile(r.tile), head(r.head), at(r.at) {}
  template <int BM, int S, int OH>
  __device__ __forceinline__ bool next(const AttnParams& p, const AttnRun& r, AttnUnit& u) {
    while (x < r.end) {
      if (read != b) {
        kv = p.kv_len[b];
        seq = attn_seq(p, p.q_offset[b], p.q_offset[b + 1], kv);
        read = b;
      }
      u.kv = kv;
      u.seq = seq;
      if (tile >= attn_tiles<BM>(seq.rows)) {
        ++b;
        tile = head = at = 0;
        continue;
      }
      u.b = b;
      u.tile = tile;
      u.head = head;
      u.row0 = tile * BM;
      u.rows = min(BM, u.seq.rows - u.row0);
      u.range = attn_tile_range<BM>(p, u.seq, u.kv, tile);
      u.n = attn_slices<S>(u.range);
      const int take = (int)min((int64_t)(OH + u.n - at), r.end - x);
      u.s0 = max(0, at - OH);
      u.s1 = max(0, at + take - OH);
      u.first = x - at + OH;
      x += take;
      at = 0;
      if (++head == p.kv_heads) {
        head = 0;
        ++tile;
      }
      if (u.s0 < u.s1) return true;  // (a run may end in front of slice 0)
    }
    return false;
  }
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool use) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(use ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
template <typename T>
__device__ __forceinline__ bool any_nonfinite(uint4 v) {
  constexpr uint32_t E = std::is_same_v<T, __nv_bfloat16> ? 0x7F80u : 0x7C00u;
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  bool bad = false;
#pragma unroll
  for (int i = 0; i < 4; ++i) bad |= (w[i] & E) == E || ((w[i] >> 16) & E) == E;
  return bad;
}

// 2^x to 2 ulp (ex2.approx): what is rounded to 8 or 11 bits, or summed, afterwards.
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// The exponent's base: a row without a finite score so far has maximum -infinity, and exponentials of 0.
__device__ __forceinline__ float safe_max(float m) { return m == -INFINITY ? 0.0f : m; }
// Weights are 2^(score - base). fp16 has them 2^7 times as large, which the division by their sum takes back: with a maximum
// that may lag by 2^8 they stay at or below 2^15 (fp16 ends at 65504), and down to 2^-21 of the largest they are normal numbers.
// Smaller ones are off by at most 2^-32 of the largest each, n keys together by n 2^-32 of the greatest |v|. bf16 has fp32's
// exponents and needs none.
template <typename T>
constexpr float kWeightShift = std::is_same_v<T, __half> ? 7.0f : 0.0f;
template <typename T>
__device__ __forceinline__ float weight_base(float m, float scale_log2) {
  if constexpr (kWeightShift<T> == 0.0f) return safe_max(m) * scale_log2;
  else return fmaf(safe_max(m), scale_log2, -kWeightShift<T>);
}
// m scale + ln of the sum of e^(score - m): `sum` is that of the weights.
template <typename T>
__device__ __forceinline__ float weights_lse(float m, float scale, float sum) {
  if constexpr (kWeightShift<T> != 0.0f) sum *= 0x1p-7f;
  return fmaf(m, scale, logf(sum));
}

// attntile.cu: 256-row units on the tensor cores, head_dim up to 128, on nsm CTAs
fp4moe_status attn_tile_launch(int32_t dtype, const AttnParams& p, int nsm, cudaStream_t st);

}  // namespace fp4moe
