// Rotary positions of q and k, and k and v into the paged cache (fp4moe_rope_cache).
//
// The pass moves (q_heads + 2 kv_heads) head_dim elements a token in and out and is bound by memory. The angle's cosine
// and sine are one for all heads of a token: a CTA makes those of its tokens once, in shared memory.
//
// Angles. turns = position * inv_freq / (2 pi) matters modulo 1 only, and a product of 64-bit integers is a product
// modulo 2^64: with step = inv_freq / (2 pi) as a fraction of 2^64, position * step is the fraction of a turn, off by
// position * 2^-53 of it at most (the rounding of step). Its upper 32 bits go to sincospif. An fp32 product would be a
// whole radian off past 2^24 radians; an fp64 sine costs a hundred fp64 operations.
//
// A thread keeps one item of a token's row (a 16-byte vector, or the two vectors that hold eight pairs of the half
// layout) and goes through the CTA's tokens with it, so places are worked out once.
#include "paged.cuh"

namespace fp4moe {
namespace {

constexpr int RC_THREADS = 256;
constexpr int RC_TOKENS = 16;  // most tokens of a CTA

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

// Cosines and sines of the CTA's tokens, and where their rows go: -1 nowhere, -2 only q.
__device__ __forceinline__ void rope_tokens(const RopeParams& p, int t0, int n, float2* cs, int64_t* at) {
  const int half = p.rot / 2;
  for (int i = threadIdx.x; i < n * half; i += RC_THREADS) {
    const int t = i / half, f = i - t * half;
    cs[t * half + f] = turn(__ldg(p.position + t0 + t), turn_step(__ldg(p.inv_freq + f)), p.amplitude);
  }
  if (threadIdx.x < n) {
    const int32_t slot = __ldg(p.slot + t0 + threadIdx.x);
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
    at[threadIdx.x] = a;
  }
  __syncthreads();
}

// Any part of the head, either layout: 16-byte vectors, each turned element's partner out of shared memory.
template <typename T>
__global__ void __launch_bounds__(RC_THREADS) rope_any_kernel(RopeParams p) {
  extern __shared__ __align__(16) uint8_t sm[];
  const int half = p.rot / 2, NV = p.D / 8;
  T* row = reinterpret_cast<T*>(sm);
  int64_t* at = reinterpret_cast<int64_t*>(sm + RC_THREADS * 16);
  float2* cs = reinterpret_cast<float2*>(at + RC_TOKENS);
  const int t0 = blockIdx.x * p.tokens, n = min(p.tokens, p.T - t0);
  pdl_wait();
  pdl_trigger();
  rope_tokens(p, t0, n, cs, at);
  const int heads = RC_THREADS / NV;  // of a CTA
  const int local = threadIdx.x / NV, d0 = (threadIdx.x - local * NV) * 8;
  const int head = blockIdx.y * heads + local;
  const int kind = head < p.q_heads ? 0 : head < p.q_heads + p.kv_heads ? 1 : 2;
  const bool live = local < heads && head < p.q_heads + 2 * p.kv_heads && (kind == 0 || p.k != nullptr);
  const int h = head - (kind > 0) * p.q_heads - (kind > 1) * p.kv_heads;
  const T* src = static_cast<const T*>(kind == 0 ? p.q : kind == 1 ? p.k : p.v);
  const int64_t stride = kind == 0 ? p.q_stride : kind == 1 ? p.k_stride : p.v_stride;
  for (int t = 0; t < n; ++t) {
    uint4 raw = make_uint4(0, 0, 0, 0);
    const int64_t a = at[t];
    const bool use = live && (kind == 0 ? a != -1 : a >= 0);
    if (use) raw = *reinterpret_cast<const uint4*>(src + (int64_t)(t0 + t) * stride + (int64_t)h * p.D + d0);
    *reinterpret_cast<uint4*>(row + threadIdx.x * 8) = raw;
    __syncthreads();
    if (use) {
      if (kind < 2) {
        T* x = reinterpret_cast<T*>(&raw);
        const T* mine = row + local * NV * 8;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int r = d0 + e - p.first;
          if (r < 0 || r >= p.rot) continue;
          const bool second = p.interleaved ? (r & 1) : r >= half;
          const int f = p.interleaved ? r >> 1 : second ? r - half : r;
          const int other = p.interleaved ? r ^ 1 : second ? r - half : r + half;
          const float2 w = cs[t * half + f];
          const float o = to_f32(mine[p.first + other]) * w.y;
          x[e] = from_f32<T>(fmaf(to_f32(x[e]), w.x, second ? o : -o));
        }
      }
      T* dst = kind == 0 ? static_cast<T*>(p.q_out) + (int64_t)(t0 + t) * p.q_out_stride + (int64_t)h * p.D
                         : static_cast<T*>(kind == 1 ? p.k_cache : p.v_cache) + a + (int64_t)h * p.map.head_stride;
      *reinterpret_cast<uint4*>(dst + d0) = raw;
    }
    __syncthreads();
  }
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
  const int per = RC_THREADS / (c.head_dim / 8);
  const int heads = q_heads + (k != nullptr ? 2 * c.kv_heads : 0), slices = (heads + per - 1) / per;
  p.tokens = (int)std::min<int64_t>(RC_TOKENS, ((int64_t)T * slices + 8 * nsm - 1) / (8 * nsm));
  const dim3 grid((unsigned)((T + p.tokens - 1) / p.tokens), (unsigned)slices);
  const size_t smem = (size_t)p.tokens * (rot_dim / 2) * 8 + RC_TOKENS * 8 + RC_THREADS * 16;
  const cudaError_t e = c.dtype == FP4MOE_BF16 ? launch_pdl(rope_any_kernel<__nv_bfloat16>, grid, dim3(RC_THREADS), smem, st, p)
                                               : launch_pdl(rope_any_kernel<__half>, grid, dim3(RC_THREADS), smem, st, p);
  return e == cudaSuccess ? FP4MOE_OK : FP4MOE_CUDA_ERROR;
}

}  // namespace fp4moe
