// Attention over the paged cache for few rows a sequence and kv head (fp4moe_paged_attention): decoding, proposed tokens.
//
// One pass over the keys: with the running maximum m and sum l of a row, each group of 16 keys (32 with 64 dims) adds
//   m' = max(m, max s), l' = l 2^(m - m') + sum 2^(s - m'), O' = O 2^(m - m') + sum 2^(s - m') v    (s in powers of two),
// where m' stays m until a score passes it by more than 2^8, so that the rows' maxima need not be made for every group.
// The bytes of k and v bound it: 16 rows of a tile cost 64 KFLOP for 8 KB of a group (head_dim 128), far below what
// mma.sync gives, so the tile's M = 16 is that of mma.sync, and a warp works alone: it brings its own groups of keys by
// cp.async through a ring of its own, without any barrier between warps, and joins the others at the end of a tile only.
// 64 sequences of up to 8192 keys, 8 kv heads of 128 dims: 1367 MB in 213 us, 6.4 TB/s, 95 % of a plain copy's rate; four of
// 131072 keys 321 us, 99 %. One row of 4096 keys is 13 us of latency: the division 2, page and keys 2, the joins 4.
// Tiles of 32 rows (64 dims) use what is read twice: 16 x 32 rows of up to 8192 keys, 8 kv heads, in 42 us, which tiles of
// 16 take 50 for and the larger ones 55. There the chain of a group binds it, scores to weights to sums, with two warps a
// scheduler to hide it: groups of 32 keys, twice as many products side by side, took it from 49 to 42 us, and decoding from
// 125 to 123; twice as many warps instead, with less of the ring and of the registers each, 52 and 128.
// Any page size and stride: a lane works out its key's place and hands it to the lanes that copy the key's 16-byte
// pieces; the page of the next group is looked up a group ahead.
// Keys outside the tile's range are zeros in shared memory. Keys that only some rows of a tile see have score -infinity
// in the others; where such a v is not finite (0 times it would be NaN) the group's product is made without those rows.
#include "attn.cuh"

namespace fp4moe {
namespace {

constexpr float AD_GROWTH = 8.0f;  // powers of two that a maximum may lag behind
constexpr int AD_MIN = 1;    // least cost of a CTA's run
constexpr int AD_OH = 1;     // what a tile costs, in slices, beside its slices

template <int DP, int RT>  // RT: 16-row MMA tiles of a tile
struct AttnCfg {
  static constexpr int kRows = 16 * RT;
  static constexpr int KT = DP == 64 ? 2 : 1, kKeys = 16 * KT;  // keys of a warp's group: 8 KB of k and v
  static constexpr int kWarps = 8;
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int S = kKeys * kWarps;           // keys of a slice: one group a warp
  static constexpr int kTile = kKeys * DP * 2;       // k, or v, of a group
  // A load is both of them (64 dims: 104 us, one at a time 121; 32 sequences of 8192 keys), or one where three of both do
  // not fit (256 dims: 343 us, both with half the warps 500).
  static constexpr int kParts = DP == 256 ? 1 : 2;
  static constexpr int kLoad = kParts * kTile;
  static constexpr int kLoads = 196608 / (kWarps * kLoad);
  static constexpr int kRing = kLoads * kLoad;         // of a warp
  static constexpr int kRings = kWarps * kRing;
  static constexpr bool kSharedQ = DP * RT >= 256;     // its 64 registers a thread are not there
  static constexpr int kSmem = kRings + (kSharedQ ? kRows * DP * 2 : 0);
  static constexpr int kPitch = DP + 8;                // floats between rows of a warp's sums: no bank conflicts
  static_assert(kLoads >= 3, "two loads under way while one is used");
  static_assert(kRows * kPitch * 4 <= kRing, "sums fit the ring");
  static_assert((FP4MOE_KV_MAX_SEQS + kWarps + 1) * 8 <= kSmem, "the division's sums fit");
};

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
template <typename T>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (std::is_same_v<T, __nv_bfloat16>)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <typename T, int DP, int RT>
__global__ void __launch_bounds__(AttnCfg<DP, RT>::kThreads, 1) attn_rows_kernel(AttnParams p) {
  using C = AttnCfg<DP, RT>;
  constexpr int ROWS = C::kRows, KEYS = C::kKeys, KT = C::KT, RL = 2 * RT;  // rows of a tile, and of a lane: qr + 8 i
  constexpr int CH = DP / 8, KS = DP / 16, NT = DP / 8;  // 16-byte pieces of a key, MMA steps, output columns of 8
  constexpr int RPI = 32 / CH;                           // keys that one copy instruction of the warp covers
  extern __shared__ __align__(1024) uint8_t sm[];
  __shared__ float stats[C::kWarps][ROWS][2];
  __shared__ uint32_t arrived, skip;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_wait();
  pdl_trigger();
  if (tid == 0) skip = *(volatile uint32_t*)p.err & kAbortMask;
  const AttnRun run = attn_plan<ROWS, C::S, AD_OH, AD_MIN, C::kThreads>(p, reinterpret_cast<int64_t*>(sm));
  if (skip) return;  // an earlier call gave up
  uint8_t* ring = sm + warp * C::kRing;
  const uint32_t ring32 = smem_u32(ring);
  const T* kbase = static_cast<const T*>(p.k);
  const T* vbase = static_cast<const T*>(p.v);
  const int dims = (p.D + 15) / 16 * 16;  // MMA steps past the head's own dims are left out
  const int qr = lane >> 2, qc = (lane & 3) * 2;
  AttnWalk walk(run);
  for (AttnUnit u; walk.next<ROWS, C::S, AD_OH>(p, run, u);) {
    const AttnSeq& seq = u.seq;
    const int kv = u.kv, head = u.head, row0 = u.row0, rows = u.rows, n = u.n, s0 = u.s0, s1 = u.s1;
    const int2 range = u.range;
    const int base = range.x / C::S * C::S + warp * KEYS;  // first key of this warp's group of slice 0
    const int32_t* table = p.table + (int64_t)u.b * p.columns;
    const int64_t head_off = (int64_t)head * p.map.head_stride;
    auto page_of = [&](int s) {  // page of the key that this lane looks up in slice s; -2: none
      const int key = base + s * C::S + (lane & (KEYS - 1));
      return s < s1 && key >= range.x && key < range.y ? table[p.map.page.div(key)] : -2;
    };
    int page = page_of(s0);  // on its way while q is fetched
    // ---- this lane's rows: q as the MMA's A, and the keys they see
    uint32_t qa[RT][C::kSharedQ ? 1 : KS][4];
    int2 see[RL];
#pragma unroll
    for (int i = 0; i < RL; ++i) {
      const int r = row0 + min(qr + 8 * i, rows - 1);  // rows past the last are computed with it, and dropped
      const int tok = (int)p.group.div(r), g = r - tok * (int)p.group.d;
      see[i] = attn_range(p, seq, kv, tok);
      const T* q = static_cast<const T*>(p.q) + (int64_t)(seq.first + tok) * p.q_stride +
                   (int64_t)(head * (int)p.group.d + g) * p.D + qc;
      if constexpr (!C::kSharedQ) {
#pragma unroll
        for (int ks = 0; ks < KS; ++ks)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int d = ks * 16 + 8 * j;
            qa[i / 2][ks][i % 2 + 2 * j] = d < p.D ? *reinterpret_cast<const uint32_t*>(q + d) : 0u;
          }
      }
    }
    if constexpr (C::kSharedQ) {  // (free since the end of the unit before)
      for (int i = tid; i < ROWS * CH; i += C::kThreads) {
        const int r = row0 + min(i / CH, rows - 1), c = i % CH, tok = (int)p.group.div(r), g = r - tok * (int)p.group.d;
        const T* q = static_cast<const T*>(p.q) + (int64_t)(seq.first + tok) * p.q_stride +
                     (int64_t)(head * (int)p.group.d + g) * p.D + c * 8;
        *reinterpret_cast<uint4*>(sm + C::kRings + (i / CH) * (DP * 2) + ((c ^ ((i / CH) & 7)) << 4)) =
            c * 8 < p.D ? *reinterpret_cast<const uint4*>(q) : make_uint4(0u, 0u, 0u, 0u);
      }
      __syncthreads();
    }
    // keys that every row of the tile sees
    const int all_lo = attn_range(p, seq, kv, (int)p.group.div(row0 + rows - 1)).x;
    const int all_hi = attn_range(p, seq, kv, (int)p.group.div(row0)).y;
    float m[RL], l[RL], o[RT][NT][4] = {};
#pragma unroll
    for (int i = 0; i < RL; ++i) {
      m[i] = -INFINITY;
      l[i] = 0.0f;
    }

    // Loads in order: of slice s0 + i for the i-th, or k, v, k, v ..
    int64_t off = -1;  // of this lane's key, in the slice whose k was issued last
    int issued = 0, fill = 0;
    auto issue = [&] {
      const int s = C::kParts == 2 ? s0 + issued : s0 + issued / 2;
      if (s < s1) {
        if (C::kParts == 2 || issued % 2 == 0) {
          const int key = base + s * C::S + (lane & (KEYS - 1));
          off = -1;
          if (page != -2) {
            if ((uint32_t)page < (uint32_t)p.map.num_pages) {
              off = page * p.map.page_stride +
                    (int64_t)(key - (int)p.map.page.div(key) * (int)p.map.page.d) * p.map.token_stride + head_off;
            } else {
              raise_error(p.err, FP4MOE_ERR_PAGE);
            }
          }
          page = page_of(s + 1);  // a group ahead
        }
        const T* from = C::kParts == 1 && issued % 2 ? vbase : kbase;
        const int c = lane % CH;
        const uint32_t dst0 = ring32 + fill * C::kLoad;
#pragma unroll
        for (int it = 0; it < KEYS / RPI; ++it) {
          const int r = it * RPI + lane / CH;
          const int64_t ro = __shfl_sync(0xFFFFFFFFu, off, r);
          const bool use = ro >= 0 && c * 8 < p.D;
          const int64_t src = use ? ro + c * 8 : 0;
          const uint32_t dst = dst0 + r * (DP * 2) + ((c ^ (r & 7)) << 4);
          if (c * 8 < dims) {
            cp_async16(dst, from + src, use);
            if (C::kParts == 2) cp_async16(dst + C::kTile, vbase + src, use);
          }
        }
      }
      cp_async_commit();
      ++issued;
      fill = fill + 1 == C::kLoads ? 0 : fill + 1;
    };
    for (int i = 0; i < C::kLoads - 1; ++i) issue();
    int stage = 0;
    auto step = [&] { stage = stage + 1 == C::kLoads ? 0 : stage + 1; };
    for (int s = s0; s < s1; ++s) {
      cp_async_wait<C::kLoads - 2>();
      __syncwarp();
      const int k0 = base + s * C::S;
      const bool any = k0 < range.y && k0 + KEYS > range.x;
      float pr[RT][2 * KT][4];
      const bool edge = k0 < all_lo || k0 + KEYS > all_hi;
      if (any) {
        const uint32_t kst = ring32 + stage * C::kLoad;
        float sc[RT][2 * KT][4] = {};
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          if (ks * 16 < dims) {
#pragma unroll
            for (int kt = 0; kt < KT; ++kt) {
              uint32_t f[4];
              const int key = kt * 16 + (lane >> 4) * 8 + (lane & 7), c = ks * 2 + ((lane >> 3) & 1);
              ldsm4(f, kst + key * (DP * 2) + ((c ^ (key & 7)) << 4));
#pragma unroll
              for (int rt = 0; rt < RT; ++rt) {
                if constexpr (C::kSharedQ) {
                  const int r = lane & 15, qc16 = ks * 2 + (lane >> 4);
                  ldsm4(qa[rt][0], smem_u32(sm) + C::kRings + (rt * 16 + r) * (DP * 2) + ((qc16 ^ (r & 7)) << 4));
                }
                mma16816<T>(sc[rt][2 * kt], qa[rt][C::kSharedQ ? 0 : ks], f[0], f[1]);
                mma16816<T>(sc[rt][2 * kt + 1], qa[rt][C::kSharedQ ? 0 : ks], f[2], f[3]);
              }
            }
          }
        }
        if (edge) {
#pragma unroll
          for (int i = 0; i < RL; ++i)
#pragma unroll
            for (int e = 0; e < 4 * KT; ++e) {
              const int key = k0 + (e >> 1) * 8 + qc + (e & 1);
              if (key < see[i].x || key >= see[i].y) sc[i / 2][e >> 1][2 * (i % 2) + (e & 1)] = -INFINITY;
            }
        }
        float nm[RL];
        bool grown = false;
#pragma unroll
        for (int i = 0; i < RL; ++i) {
          nm[i] = -INFINITY;  // of this lane's keys
#pragma unroll
          for (int t = 0; t < 2 * KT; ++t) nm[i] = fmaxf(nm[i], fmaxf(sc[i / 2][t][2 * (i % 2)], sc[i / 2][t][2 * (i % 2) + 1]));
          grown |= (nm[i] - m[i]) * p.scale_log2 > AD_GROWTH;
        }
        if (__any_sync(0xFFFFFFFFu, grown)) {
#pragma unroll
          for (int i = 0; i < RL; ++i) {
            nm[i] = fmaxf(nm[i], __shfl_xor_sync(0xFFFFFFFFu, nm[i], 1));
            nm[i] = fmaxf(nm[i], __shfl_xor_sync(0xFFFFFFFFu, nm[i], 2));
            nm[i] = fmaxf(m[i], nm[i]);
            const float f = exp2_fast((m[i] - safe_max(nm[i])) * p.scale_log2);
            l[i] *= f;
#pragma unroll
            for (int t = 0; t < NT; ++t) {
              o[i / 2][t][2 * (i % 2)] *= f;
              o[i / 2][t][2 * (i % 2) + 1] *= f;
            }
            m[i] = nm[i];
          }
        }
#pragma unroll
        for (int i = 0; i < RL; ++i) {
          const float mb = weight_base<T>(m[i], p.scale_log2);
#pragma unroll
          for (int t = 0; t < 2 * KT; ++t)
#pragma unroll
            for (int e = 2 * (i % 2); e < 2 * (i % 2) + 2; ++e) {
              pr[i / 2][t][e] = exp2_fast(fmaf(sc[i / 2][t][e], p.scale_log2, -mb));
              l[i] += pr[i / 2][t][e];
            }
        }
      }
      if constexpr (C::kParts == 1) {
        __syncwarp();
        issue();
        step();
        cp_async_wait<C::kLoads - 2>();
        __syncwarp();
      }
      if (any) {
        const uint8_t* vt = ring + stage * C::kLoad + (C::kParts - 1) * C::kTile;
        const uint32_t vst = ring32 + stage * C::kLoad + (C::kParts - 1) * C::kTile;
        bool odd = false;  // a v that some rows must not touch even with weight 0
        if (edge && (all_lo != range.x || all_hi != range.y)) {
          for (int it = 0; it < KEYS / RPI; ++it) {
            const int r = it * RPI + lane / CH, c = lane % CH;
            if (c * 8 < dims)
              odd |= any_nonfinite<T>(
                  *reinterpret_cast<const uint4*>(vt + r * (DP * 2) + ((c ^ (r & 7)) << 4)));
          }
          odd = __any_sync(0xFFFFFFFFu, odd);
        }
        if (!odd) {
          // the weights are rounded to the cache's type for the MMA: half a step each, against a result of that type
#pragma unroll
          for (int kt = 0; kt < KT; ++kt) {
            uint32_t pa[RT][4];
#pragma unroll
            for (int rt = 0; rt < RT; ++rt)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float(&w)[4] = pr[rt][2 * kt + (e >> 1)];
                pa[rt][e] = pack2<T>(w[2 * (e & 1)], w[2 * (e & 1) + 1]);
              }
#pragma unroll
            for (int t = 0; t < NT; t += 2) {
              if (t * 8 < dims) {
                uint32_t f[4];
                const int key = kt * 16 + ((lane >> 3) & 1) * 8 + (lane & 7), c = t + (lane >> 4);
                ldsm4_t(f, vst + key * (DP * 2) + ((c ^ (key & 7)) << 4));
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) {
                  mma16816<T>(o[rt][t], pa[rt], f[0], f[1]);
                  mma16816<T>(o[rt][t + 1], pa[rt], f[2], f[3]);
                }
              }
            }
          }
        } else {
#pragma unroll 1
          for (int c = 0; c < KEYS; ++c) {
            float w[RL];
#pragma unroll
            for (int i = 0; i < RL; ++i) {
              const int at = 2 * (i % 2);
              w[i] = 0.0f;
#pragma unroll
              for (int t = 0; t < 2 * KT; ++t) {  // (all eights of keys are asked for, so that the weights stay in registers)
                const float x = __shfl_sync(0xFFFFFFFFu, (c & 1) ? pr[i / 2][t][at + 1] : pr[i / 2][t][at], (lane & ~3) + ((c & 7) >> 1));
                if (t == c >> 3) w[i] = x;
              }
            }
#pragma unroll
            for (int t = 0; t < NT; ++t) {
              if (t * 8 < dims) {
                const T* v = reinterpret_cast<const T*>(vt + c * (DP * 2) + ((t ^ (c & 7)) << 4)) + qc;
                const float v0 = to_f32(v[0]), v1 = to_f32(v[1]);
#pragma unroll
                for (int i = 0; i < RL; ++i) {
                  if (k0 + c < see[i].x || k0 + c >= see[i].y) continue;
                  float(&o4)[4] = o[i / 2][t];
                  o4[2 * (i % 2)] = fmaf(w[i], v0, o4[2 * (i % 2)]);
                  o4[2 * (i % 2) + 1] = fmaf(w[i], v1, o4[2 * (i % 2) + 1]);
                }
              }
            }
          }
        }
      }
      __syncwarp();
      issue();
      step();
    }
    cp_async_wait<0>();
    __syncwarp();
    // ---- the warps' sums, in their rings
    float* mine = reinterpret_cast<float*>(ring);
#pragma unroll
    for (int i = 0; i < RL; ++i) {
      l[i] += __shfl_xor_sync(0xFFFFFFFFu, l[i], 1);
      l[i] += __shfl_xor_sync(0xFFFFFFFFu, l[i], 2);
      if ((lane & 3) == 0) {
        stats[warp][qr + 8 * i][0] = m[i];
        stats[warp][qr + 8 * i][1] = l[i];
      }
#pragma unroll
      for (int t = 0; t < NT; ++t)
        *reinterpret_cast<float2*>(mine + (qr + 8 * i) * C::kPitch + t * 8 + qc) = make_float2(o[i / 2][t][2 * (i % 2)], o[i / 2][t][2 * (i % 2) + 1]);
    }
    __syncthreads();
    constexpr int TPR = C::kThreads / ROWS, NJ = DP / (4 * TPR);  // threads of a row, vectors of a thread
    const int r = tid / TPR, dv = (tid % TPR) * 4;
    float M = -INFINITY, L = 0.0f;
    float4 acc[NJ];
#pragma unroll
    for (int j = 0; j < NJ; ++j) acc[j] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int w = 0; w < C::kWarps; ++w) M = fmaxf(M, stats[w][r][0]);
#pragma unroll
    for (int w = 0; w < C::kWarps; ++w) {
      const float f = exp2_fast((stats[w][r][0] - safe_max(M)) * p.scale_log2);
      L = fmaf(stats[w][r][1], f, L);
      const float* src = reinterpret_cast<const float*>(sm + w * C::kRing) + r * C::kPitch + dv;
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const float4 v = *reinterpret_cast<const float4*>(src + j * 4 * TPR);
        acc[j].x = fmaf(v.x, f, acc[j].x);
        acc[j].y = fmaf(v.y, f, acc[j].y);
        acc[j].z = fmaf(v.z, f, acc[j].z);
        acc[j].w = fmaf(v.w, f, acc[j].w);
      }
    }
    bool whole = s0 == 0 && s1 == n;
    if (!whole) {
      const int c0 = attn_owner(run, u.first), c1 = attn_owner(run, u.first + n - 1);
      float2* st = reinterpret_cast<float2*>(p.ws + kAttnStats);
      float* sums = reinterpret_cast<float*>(p.ws + kAttnSums);
      const int64_t slot = 2 * blockIdx.x + (s0 == 0);
      if (r < rows) {
        if (dv == 0) __stcg(st + slot * ROWS + r, make_float2(M, L));
#pragma unroll
        for (int j = 0; j < NJ; ++j)
          __stcg(reinterpret_cast<float4*>(sums + (slot * ROWS + r) * DP + dv + j * 4 * TPR), acc[j]);
      }
      __syncthreads();
      if (tid == 0) {  // its fences stand for the CTA's writes before the barrier, and for its reads after the next
        uint32_t* count = reinterpret_cast<uint32_t*>(p.ws + kAttnCounters) + 2 * c0;
        __threadfence();
        arrived = atomicAdd(count, 1u);
        __threadfence();
        if (arrived == (uint32_t)(c1 - c0)) *count = 0;
      }
      __syncthreads();
      if (arrived == (uint32_t)(c1 - c0)) {  // the last: adds all parts in order
        whole = true;
        M = -INFINITY;
        L = 0.0f;
#pragma unroll
        for (int j = 0; j < NJ; ++j) acc[j] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (r < rows) {
#pragma unroll 8
          for (int c = c0; c <= c1; ++c) M = fmaxf(M, __ldcg(st + (int64_t)(2 * c + (c == c0)) * ROWS + r).x);
#pragma unroll 4
          for (int c = c0; c <= c1; ++c) {
            const int64_t at = (int64_t)(2 * c + (c == c0)) * ROWS + r;
            const float2 ml = __ldcg(st + at);
            const float f = exp2_fast((ml.x - safe_max(M)) * p.scale_log2);
            L = fmaf(ml.y, f, L);
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
              const float4 v = __ldcg(reinterpret_cast<const float4*>(sums + at * DP + dv + j * 4 * TPR));
              acc[j].x = fmaf(v.x, f, acc[j].x);
              acc[j].y = fmaf(v.y, f, acc[j].y);
              acc[j].z = fmaf(v.z, f, acc[j].z);
              acc[j].w = fmaf(v.w, f, acc[j].w);
            }
          }
        }
      }
    }
    if (whole && r < rows) {
      const int tok = (int)p.group.div(row0 + r), g = row0 + r - tok * (int)p.group.d;
      const int2 sees = attn_range(p, seq, kv, tok);
      // a row without keys is 0; one whose scores are all -infinity is 0 / 0
      const float inv = sees.x < sees.y ? __fdiv_rn(1.0f, L) : 0.0f;
      const bool none = sees.x >= sees.y;
      const int64_t t = seq.first + tok;
      const int hq = head * (int)p.group.d + g;
      T* out = static_cast<T*>(p.out) + t * p.out_stride + (int64_t)hq * p.D;
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const int d = dv + j * 4 * TPR;
        if (d < p.D) {
          const uint2 v = none ? make_uint2(0u, 0u)
                               : make_uint2(pack2<T>(acc[j].x * inv, acc[j].y * inv), pack2<T>(acc[j].z * inv, acc[j].w * inv));
          *reinterpret_cast<uint2*>(out + d) = v;
        }
      }
      if (p.lse != nullptr && dv == 0) p.lse[t * p.q_heads + hq] = none ? -INFINITY : weights_lse<T>(M, p.scale, L);
    }
    __syncthreads();
  }
}

template <typename T, int DP, int RT>
fp4moe_status attn_rows_run(const AttnParams& p, int nsm, cudaStream_t st) {
  using C = AttnCfg<DP, RT>;
  static PerDevice done;
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return FP4MOE_CUDA_ERROR;
  if (done.get(dev, [] {
        return cudaFuncSetAttribute(attn_rows_kernel<T, DP, RT>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem) ==
                       cudaSuccess
                   ? 1
                   : 0;
      }) <= 0)
    return FP4MOE_CUDA_ERROR;
  return launch_pdl(attn_rows_kernel<T, DP, RT>, dim3((unsigned)nsm), dim3(C::kThreads), C::kSmem, st, p) == cudaSuccess
             ? FP4MOE_OK
             : FP4MOE_CUDA_ERROR;
}
template <typename T>
fp4moe_status attn_rows_typed(const AttnParams& p, int tile, int nsm, cudaStream_t st) {
  return tile == 32   ? attn_rows_run<T, 64, 2>(p, nsm, st)
         : p.D <= 64  ? attn_rows_run<T, 64, 1>(p, nsm, st)
         : p.D <= 128 ? attn_rows_run<T, 128, 1>(p, nsm, st)
                      : attn_rows_run<T, 256, 1>(p, nsm, st);
}

}  // namespace

// Sequences of more than 16 rows a kv head, on the average, are for larger tiles, which read k and v once for more rows,
// unless all of them are a few tiles of 16, which a part of the SMs works on. Heads of 32 / 8, us with tiles of 16, 32, 256:
//   128 dims, 16 sequences of up to 8192 keys: 16 rows 62, 78, 71; 32 rows 91, 80, 72; one sequence of 8192: 32 rows 22, 21,
//   28, 48 rows 26, 27, 56. Tiles of 32 gain too little there to be kept.
//   64 dims, 16 sequences of up to 8192 keys: 16 rows 38, 41, 54; 32 rows 53, 43, 56; 48 rows 75, 60, 56; one sequence of
//   8192: 32 rows 14, 15, 25, 64 rows 20, 16, 36.
// Those are sequences of one length. The average decides for unequal ones too: 512 decodes beside one chunk of 1500 tokens,
// 5000 keys each, 128 dims, go through tiles of 16 in 2006 us, 64 beside a chunk of 1024 through the larger ones in 314. Decodes
// and chunks in calls of their own take 1507 + 90 and 202 + 73.
int paged_attention_tile(const fp4moe_kv_cache& c, int32_t num_seqs, int32_t T, int32_t q_heads) {
  const int64_t rows = (int64_t)T * (q_heads / c.kv_heads), tiles = (rows + 15) / 16 * c.kv_heads;
  if (num_seqs == 0 || c.head_dim > 128 || rows <= (int64_t)16 * num_seqs) return 16;
  if (c.head_dim > 64) return tiles > 48 ? kAttnTileRows : 16;
  return tiles > 48 && rows > (int64_t)32 * num_seqs ? kAttnTileRows : 32;
}

fp4moe_status paged_attention_launch(const fp4moe_kv_cache& c, const void* k_cache, const void* v_cache, int32_t num_seqs,
                                     int32_t T, int32_t q_heads, const void* q, int64_t q_stride,
                                     const int32_t* page_table, int32_t table_columns, const int32_t* kv_len,
                                     const int32_t* q_offset, float scale, bool causal, int32_t window, void* out,
                                     int64_t out_stride, float* lse, void* ws, uint32_t* err, cudaStream_t st) {
  AttnParams p{};
  p.map = cache_map(c);
  p.k = k_cache;
  p.v = v_cache;
  p.q = q;
  p.out = out;
  p.lse = lse;
  p.table = page_table;
  p.kv_len = kv_len;
  p.q_offset = q_offset;
  p.q_stride = q_stride;
  p.out_stride = out_stride;
  p.B = num_seqs;
  p.T = T;
  p.q_heads = q_heads;
  p.kv_heads = c.kv_heads;
  p.D = c.head_dim;
  p.columns = table_columns;
  p.group = FastDiv((uint32_t)(q_heads / c.kv_heads));
  p.causal = causal;
  p.window = window;
  p.scale = scale;
  p.scale_log2 = scale * 1.44269504088896340736f;
  p.ws = static_cast<uint8_t*>(ws);
  p.err = err;
  int nsm = sm_count();
  if (nsm <= 0) return FP4MOE_CUDA_ERROR;
  if (nsm > kAttnMaxCtas) nsm = kAttnMaxCtas;
  const int tile = paged_attention_tile(c, num_seqs, T, q_heads);
  if (tile == kAttnTileRows) return attn_tile_launch(c.dtype, p, nsm, st);
  return c.dtype == FP4MOE_BF16 ? attn_rows_typed<__nv_bfloat16>(p, tile, nsm, st) : attn_rows_typed<__half>(p, tile, nsm, st);
}

}  // namespace fp4moe
