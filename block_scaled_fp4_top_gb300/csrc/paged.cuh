// The paged key-value cache as its kernels see it (kvplan.cu, rope.cu, attn.cu, attntile.cu).
// They start before the kernel in front of them has ended, and lengths may be outputs too: what the calls write is read with
// plain loads, behind pdl_wait, since read-only loads (__ldg) are for memory that does not change while a kernel lives.
#pragma once

#include "dense.cuh"
#include "internal.h"
#include "perdevice.h"

namespace fp4moe {

// n / d for 0 <= n < 2^31 by a multiplication: with m = ceil(2^p / d), p = 31 + ceil(log2 d), n m / 2^p exceeds n / d
// by less than n / 2^p <= 1 / d, so the floor is that of n / d.
struct FastDiv {
  uint32_t d, m, p;
  __host__ __device__ FastDiv() : d(1), m(1u << 31), p(31) {}
  explicit FastDiv(uint32_t div) : d(div), p(31) {
    while ((1ull << (p - 31)) < d) ++p;
    m = (uint32_t)(((1ull << p) + d - 1) / d);
  }
  __device__ __forceinline__ uint32_t div(uint32_t n) const { return (uint32_t)(((uint64_t)n * m) >> p); }
};

// Element offset of a token of the cache, kv head 0.
struct CacheMap {
  FastDiv page;
  int num_pages;
  int64_t page_stride, token_stride, head_stride;
};
inline CacheMap cache_map(const fp4moe_kv_cache& c) {
  CacheMap m;
  m.page = FastDiv((uint32_t)c.page_size);
  m.num_pages = c.num_pages;
  m.page_stride = c.page_stride;
  m.token_stride = c.token_stride;
  m.head_stride = c.head_stride;
  return m;
}

}  // namespace fp4moe
