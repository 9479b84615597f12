// Rotary positions of q and k, and k and v into the paged cache (fp4moe_rope_cache).
//
// The pass moves (q_heads + 2 kv_heads) head_dim elements a token in and out and is bound by memory: 8192 tokens of 32 + 8 + 8
// heads of 128 dims, 201 MB in and out, in 34.4 us, 5.9 TB/s. The angle's cosine and sine are one for all heads of a token: a
// CTA makes those of its tokens once, in shared memory, and a token's row has CTAs of its own where there are few.
//
// Angles. turns = position * inv_freq / (2 pi) matters modulo 1 only, and a product of 64-bit integers is a product
// modulo 2^64: with step = inv_freq / (2 pi) as a fraction of 2^64, position * step is the fraction of a turn, off by
// position * |inv_freq| * 2^-55 turns at most: 1 / (2 pi) is off by 2^-53.8 of itself and the product by 2^-53, over 2 pi.
// Its upper 32 bits go to sincospif as fp32, whose 24 bits are 2^-26 turns at most of half a turn. An fp32 product would be
// a whole radian off past 2^24 radians; an fp64 sine costs a hundred fp64 operations.
//
// rope_vec_kernel: a thread keeps one item of a token's row (a 16-byte vector, or the two vectors that hold eight pairs of
// the half layout) and goes through the CTA's tokens with it, the next two on their way, so places are worked out once. It takes
// parts of the head that consist of whole vectors. rope_any_kernel takes the others: a warp has whole heads in shared
// memory, and each turned element picks its partner there, one token after the other with no load under way: 8192 tokens
// as above take 72 us with 38 dims turned and 81 with 126 in neighbouring pairs, 2.5 to 2.8 TB/s.
#include <algorithm>

#include "paged.cuh"

namespace fp4moe {
namespace {

constexpr int RC_THREADS = 256;  // of rope_any_kernel
constexpr int RC_MAX_THREADS = 512;
constexpr int RC_TOKENS = 16;    // most tokens of a CTA
constexpr int RC_UNROLL = 2;

struct RopeParams {
  int T, q_heads, kv_heads, D;
  const void *q, *k, *v;
  int64_t q_stride, k_stride, v_stride, q_out_stride;
  const int32_t *position, *slot;
  const double* inv_freq;
  int first, rot, interleaved;
  float amplitude;
  void *q_out, *k_cache, *v_cache;
  CacheMap map;
  uint32_t* err;
  int tokens;  // of a CTA
};

// inv_freq radians as a fraction of a turn, in units of 2^-64.
__device__ __forceinline__ int64_t turn_step(double inv_freq) {
  double t = inv_freq * 0.15915494309189533577;
  t -= rint(t);
  return (int64_t)(t * 0x1p63) << 1;  // |t| <= 1/2: 2^63 saturates, half a turn all the same
}
__device__ __forceinline__ float2 turn(int32_t position, int64_t step, float amplitude) {
  const int32_t part = (int32_t)(((uint64_t)(int64_t)position * (uint64_t)step) >> 32);
  float s, c;
  sincospif((float)part * 0x1p-31f, &s, &c);
  return make_float2(c * amplitude, s * amplitude);
}

// Shared memory of a CTA.
struct RopeShared {
  int64_t* at;     // [RC_TOKENS] where a token's k and v go: -1 nowhere, and its q neither; -2 nowhere, but its q does
  int64_t* step;   // [rot / 2]
  float2* turns;   // [tokens][rot / 2] cosine and sine
};
__device__ __forceinline__ RopeShared rope_shared(uint8_t* sm, int half) {
  RopeShared s;
  s.at = reinterpret_cast<int64_t*>(sm);
  s.turns = reinterpret_cast<float2*>(sm + RC_TOKENS * 8);
  s.step = reinterpret_cast<int64_t*>(sm + RC_TOKENS * 8);
  s.turns += half;  // (8 bytes each, as the steps are)
  return s;
}
inline size_t rope_shared_bytes(int tokens, int half) { return RC_TOKENS * 8 + (size_t)(tokens + 1) * half * 8; }

// Tokens [t0, t0 + n) of the CTA.
__device__ __forceinline__ void rope_tokens(const RopeParams& p, int t0, int n, const RopeShared& s) {
  const int half = p.rot / 2;
  for (int f = threadIdx.x; f < half; f += blockDim.x) s.step[f] = turn_step(__ldg(p.inv_freq + f));
  if (threadIdx.x < n) {
    const int32_t slot = p.slot[t0 + threadIdx.x];
    int64_t a = -1;
    if (slot != -1) {
      const uint32_t page = slot < 0 ? (uint32_t)p.map.num_pages : p.map.page.div((uint32_t)slot);
      if (page < (uint32_t)p.map.num_pages) {
        a = (int64_t)page * p.map.page_stride + (int64_t)((uint32_t)slot - page * p.map.page.d) * p.map.token_stride;
      } else {
        a = -2;
        if (p.k != nullptr && blockIdx.y == 0) raise_error(p.err, FP4MOE_ERR_PAGE);
      }
    }
    s.at[threadIdx.x] = a;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n * half; i += blockDim.x) {
    const int t = i / half, f = i - t * half;
    s.turns[i] = turn(p.position[t0 + t], s.step[f], p.amplitude);
  }
  __syncthreads();
}

// Where a head's elements come from and go to; k and v go to the cache.
template <typename T>
struct RopeHead {
  const T* src;
  int64_t stride, out_stride;
  T* dst;
  bool live, q;
  __device__ __forceinline__ RopeHead(const RopeParams& p, int head) {
    const int kind = head < p.q_heads ? 0 : head < p.q_heads + p.kv_heads ? 1 : 2;
    const int h = head - (kind > 0) * p.q_heads - (kind > 1) * p.kv_heads;
    q = kind == 0;
    live = head < p.q_heads + (p.k != nullptr ? 2 * p.kv_heads : 0);
    stride = kind == 0 ? p.q_stride : kind == 1 ? p.k_stride : p.v_stride;
    src = static_cast<const T*>(kind == 0 ? p.q : kind == 1 ? p.k : p.v) + (int64_t)h * p.D;
    out_stride = p.q_out_stride;
    dst = q ? static_cast<T*>(p.q_out) + (int64_t)h * p.D
            : static_cast<T*>(kind == 1 ? p.k_cache : p.v_cache) + (int64_t)h * p.map.head_stride;
  }
  __device__ __forceinline__ bool takes(int64_t at) const { return live && (q ? at != -1 : at >= 0); }
  __device__ __forceinline__ const T* from(int64_t t) const { return src + t * stride; }
  __device__ __forceinline__ T* to(int64_t t, int64_t at) const { return dst + (q ? t * out_stride : at); }
};

// Parts of the head that are whole 16-byte vectors: first, and rot / 2 (half layout) or rot (interleaved), multiples of 8.
template <typename T, bool INTERLEAVED>
__global__ void __launch_bounds__(RC_MAX_THREADS) rope_vec_kernel(RopeParams p) {
  extern __shared__ __align__(16) uint8_t sm[];
  const int half = p.rot / 2, NV = p.D / 8, turned = p.q_heads + p.kv_heads;
  const RopeShared s = rope_shared(sm, half);
  const int t0 = blockIdx.x * p.tokens, n = min(p.tokens, p.T - t0);
  // this thread's item: vectors v0 and, of the half layout's pairs, v1
  const int pairs = INTERLEAVED ? 0 : half / 8, per = NV - pairs;
  const int item = blockIdx.y * blockDim.x + threadIdx.x;
  int head, v0, v1 = -1, f = -1;  // f: first of its frequencies, -1: none
  if (item < turned * per) {
    head = item / per;
    v0 = item - head * per;
    if (INTERLEAVED) {
      if (v0 * 8 >= p.first && v0 * 8 < p.first + p.rot) f = (v0 * 8 - p.first) / 2;
    } else if (v0 < pairs) {
      f = v0 * 8;
      v0 += p.first / 8;
      v1 = v0 + pairs;
    } else {
      v0 -= pairs;
      if (v0 >= p.first / 8) v0 += 2 * pairs;
    }
  } else {
    head = turned + (item - turned * per) / NV;
    v0 = (item - turned * per) % NV;
  }
  const RopeHead<T> h(p, head);
  pdl_wait();
  pdl_trigger();
  struct Group {
    uint4 a[RC_UNROLL], b[RC_UNROLL];
  };
  auto load = [&](Group& g, int t) {  // of padding rows too: they are there
#pragma unroll
    for (int i = 0; i < RC_UNROLL; ++i) {
      if (h.live && t + i < n) {
        const uint4* src = reinterpret_cast<const uint4*>(h.from(t0 + t + i));
        g.a[i] = src[v0];
        if (!INTERLEAVED && v1 >= 0) g.b[i] = src[v1];
      }
    }
  };
  auto store = [&](Group& g, int t) {
#pragma unroll
    for (int i = 0; i < RC_UNROLL; ++i) {
      if (t + i >= n) break;
      const int64_t at = s.at[t + i];
      if (!h.takes(at)) continue;
      uint4* dst = reinterpret_cast<uint4*>(h.to(t0 + t + i, at));
      if (f >= 0) {
        const float2* w = s.turns + (t + i) * half + f;
        float x[8];
        unpack<T>(g.a[i], x);
        if constexpr (INTERLEAVED) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 c = w[e];
            const float u = x[2 * e], v = x[2 * e + 1];
            x[2 * e] = fmaf(u, c.x, -v * c.y);
            x[2 * e + 1] = fmaf(v, c.x, u * c.y);
          }
        } else {
          float y[8];
          unpack<T>(g.b[i], y);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float2 c = w[e];
            const float u = x[e], v = y[e];
            x[e] = fmaf(u, c.x, -v * c.y);
            y[e] = fmaf(v, c.x, u * c.y);
          }
          dst[v1] = pack<T>(y);
        }
        g.a[i] = pack<T>(x);
      }
      dst[v0] = g.a[i];
    }
  };
  Group now, next;
  load(now, 0);  // on their way while the cosines are made
  rope_tokens(p, t0, n, s);
  for (int t = 0; t < n; t += RC_UNROLL) {
    load(next, t + RC_UNROLL);
    store(now, t);
    now = next;
  }
}

// Any part of the head, either layout.
template <typename T>
__global__ void __launch_bounds__(RC_THREADS) rope_any_kernel(RopeParams p) {
  extern __shared__ __align__(16) uint8_t sm[];
  const int half = p.rot / 2, NV = p.D / 8, lane = threadIdx.x & 31;
  T* row = reinterpret_cast<T*>(sm) + (threadIdx.x & ~31) * 8;  // of the warp
  const RopeShared s = rope_shared(sm + RC_THREADS * 16, half);
  const int t0 = blockIdx.x * p.tokens, n = min(p.tokens, p.T - t0);
  pdl_wait();
  pdl_trigger();
  rope_tokens(p, t0, n, s);
  const int heads = 32 / NV, local = lane / NV, v = lane - local * NV;  // of a warp
  const int head = (blockIdx.y * (RC_THREADS / 32) + threadIdx.x / 32) * heads + local;
  RopeHead<T> h(p, head);
  h.live &= local < heads;
  const bool turns = head < p.q_heads + p.kv_heads;
  for (int t = 0; t < n; ++t) {
    const int64_t at = s.at[t];
    const bool use = h.takes(at);
    uint4 raw = make_uint4(0, 0, 0, 0);
    if (use) raw = reinterpret_cast<const uint4*>(h.from(t0 + t))[v];
    reinterpret_cast<uint4*>(row)[lane] = raw;
    __syncwarp();
    if (use) {
      if (turns) {
        T* x = reinterpret_cast<T*>(&raw);
        const T* mine = row + local * NV * 8 + p.first;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int r = v * 8 + e - p.first;
          if (r < 0 || r >= p.rot) continue;
          const bool second = p.interleaved ? (r & 1) : r >= half;
          const int f = p.interleaved ? r >> 1 : second ? r - half : r;
          const int other = p.interleaved ? r ^ 1 : second ? r - half : r + half;
          const float2 w = s.turns[t * half + f];
          const float o = to_f32(mine[other]) * w.y;
          x[e] = from_f32<T>(fmaf(to_f32(x[e]), w.x, second ? o : -o));
        }
      }
      reinterpret_cast<uint4*>(h.to(t0 + t, at))[v] = raw;
    }
    __syncwarp();
  }
}

template <typename T>
cudaError_t rope_launch(RopeParams p, int nsm, cudaStream_t st) {
  const int NV = p.D / 8, half = p.rot / 2, heads = p.q_heads + (p.k != nullptr ? 2 * p.kv_heads : 0);
  const bool vec = p.first % 8 == 0 && (p.interleaved ? p.rot % 8 == 0 : half % 8 == 0);
  int threads, slices;
  if (vec) {  // slices of the row's items, as even as they get
    const int turned = std::min(heads, p.q_heads + (p.k != nullptr ? p.kv_heads : 0));
    const int items = heads * NV - (p.interleaved ? 0 : turned * (half / 8));
    slices = (items + RC_MAX_THREADS - 1) / RC_MAX_THREADS;
    threads = ((items + slices - 1) / slices + 31) / 32 * 32;
  } else {
    const int per = RC_THREADS / 32 * (32 / NV);
    slices = (heads + per - 1) / per;
    threads = RC_THREADS;
  }
  // enough CTAs for every SM to hold 2048 threads, but no more tokens to one than share its cosines well
  const int64_t ctas = (int64_t)nsm * (2048 / threads);
  p.tokens = (int)std::min<int64_t>(RC_TOKENS, ((int64_t)p.T * slices + ctas - 1) / ctas);
  const dim3 grid((unsigned)((p.T + p.tokens - 1) / p.tokens), (unsigned)slices);
  const size_t smem = rope_shared_bytes(p.tokens, half);
  if (!vec) return launch_pdl(rope_any_kernel<T>, grid, dim3(threads), smem + RC_THREADS * 16, st, p);
  return p.interleaved ? launch_pdl(rope_vec_kernel<T, true>, grid, dim3(threads), smem, st, p)
                       : launch_pdl(rope_vec_kernel<T, false>, grid, dim3(threads), smem, st, p);
}

}  // namespace

fp4moe_status rope_cache_launch(const fp4moe_kv_cache& c, int32_t T, int32_t q_heads, const void* q, int64_t q_stride,
                                const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                                const int32_t* position, const int32_t* slot, int32_t rot_first, int32_t rot_dim,
                                bool interleaved, const double* inv_freq, float amplitude, void* q_out,
                                int64_t q_out_stride, void* k_cache, void* v_cache, uint32_t* err, cudaStream_t st) {
  RopeParams p{};
  p.T = T;
  p.q_heads = q_heads;
  p.kv_heads = c.kv_heads;
  p.D = c.head_dim;
  p.q = q;
  p.k = k;
  p.v = v;
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.q_out_stride = q_out_stride;
  p.position = position;
  p.slot = slot;
  p.inv_freq = inv_freq;
  p.first = rot_first;
  p.rot = rot_dim;
  p.interleaved = interleaved;
  p.amplitude = amplitude;
  p.q_out = q_out;
  p.k_cache = k_cache;
  p.v_cache = v_cache;
  p.map = cache_map(c);
  p.err = err;
  const int nsm = sm_count();
  if (nsm <= 0) return FP4MOE_CUDA_ERROR;
  return (c.dtype == FP4MOE_BF16 ? rope_launch<__nv_bfloat16>(p, nsm, st) : rope_launch<__half>(p, nsm, st)) == cudaSuccess
             ? FP4MOE_OK
             : FP4MOE_CUDA_ERROR;
}

}  // namespace fp4moe
