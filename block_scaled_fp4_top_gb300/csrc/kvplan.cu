// Page tables, positions and cache slots of a step's new tokens, from the lengths of its sequences (fp4moe_kv_plan).
//
// Three running sums over the sequences decide everything: of the new tokens (a sequence's first row), of the pages
// given back (their places on the stack) and of the pages taken. With F pages on the stack and P given back, the k-th
// page taken is entry F + P - 1 - k of the stack with the P on top, which is either an old entry or, found by a search in
// the second sum, a table entry of a sequence that gives pages back. So no step waits for another one's writes: old
// entries below F and the tables of shrinking sequences are only read, entries from F on and new columns of growing
// sequences only written. The sums cost less than a launch: every CTA of one cluster makes them all for itself in shared
// memory, then takes its share of the tokens, pages and sequences. The outputs that may lie in an input's place
// (kv_len, free_count_out) are written behind a cluster barrier, when every CTA has read the inputs.
// What bounds it is latency: 64 sequences of one new token take 4.9 us in a graph, 512 with 50000 new tokens 14.2.
#include "paged.cuh"

namespace fp4moe {
namespace {

constexpr int KP_THREADS = 1024;
constexpr int KP_ITEMS = FP4MOE_KV_MAX_SEQS / KP_THREADS;  // sequences of a thread
constexpr int KP_MAX_CLUSTER = 8;

struct KvPlanParams {
  int B, columns, num_pages, rows;
  FastDiv page;
  const int32_t *cached, *fresh;
  int32_t* table;
  int32_t* free_pages;
  const int32_t* free_count;
  int32_t *kv_len, *free_count_out, *q_offset, *position, *slot;
  uint32_t* err;
};

// Exclusive sum over the block of one value per thread, and the total; `part` holds 33 words.
__device__ __forceinline__ int64_t block_sum(int64_t v, int64_t* part, int64_t& total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  int64_t x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xFFFFFFFFu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) part[w] = x;
  __syncthreads();
  if (w == 0) {
    int64_t s = part[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xFFFFFFFFu, s, o);
      if (lane >= o) s += y;
    }
    part[lane] = s;
  }
  __syncthreads();
  total = part[31];
  const int64_t before = w ? part[w - 1] : 0;
  __syncthreads();
  return before + x - v;
}

// Last i in [0, n) with s[i] <= x, for a non-decreasing s with s[0] <= x.
__device__ __forceinline__ int last_at_most(const int32_t* s, int n, int32_t x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (s[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

__device__ __forceinline__ int32_t clamp32(int64_t v, int64_t hi) { return (int32_t)(v < hi ? v : hi); }

__global__ void __launch_bounds__(KP_THREADS) kv_plan_kernel(KvPlanParams p) {
  extern __shared__ int32_t sm[];
  const int B = p.B;
  int32_t* first = sm;               // [B + 1] a sequence's first row
  int32_t* taken = first + B + 1;    // [B] pages taken by the sequences before
  int32_t* given = taken + B;        // [B] pages given back by the sequences before
  int32_t* from = given + B;         // [B] c, or ~c if the sequence takes nothing
  int32_t* to = from + B;            // [B] a
  __shared__ int64_t part[32];
  __shared__ int first_refused;      // pages taken by the sequences before the first that the stack refused
  __shared__ uint32_t errors;
  const int tid = threadIdx.x;
  const uint32_t rank = cluster_ctarank();
  uint32_t ctas;
  asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(ctas));
  pdl_wait();
  pdl_trigger();
  // no length whose pages cannot be counted in 32 bits
  const int64_t columns = (int64_t)p.columns * p.page.d, most = (int64_t)INT32_MAX - p.page.d;
  const int64_t limit = columns < most ? columns : most;
  auto pages = [&](int32_t n) { return (int32_t)p.page.div((uint32_t)n + p.page.d - 1); };
  uint32_t err = 0;
  if (tid == 0) {
    first_refused = INT32_MAX;
    errors = 0;
  }
  // ---- lengths, first rows and pages given back
  const int per = (B + KP_THREADS - 1) / KP_THREADS, b0 = tid * per;
  int64_t tokens = 0, back = 0;
  int32_t fresh[KP_ITEMS];
#pragma unroll
  for (int i = 0; i < KP_ITEMS; ++i) {
    const int b = b0 + i;
    if (i >= per || b >= B) break;
    int64_t c = p.cached[b];
    const int64_t n = fresh[i] = p.fresh[b];
    if (c < 0 || c > limit) {
      err |= FP4MOE_ERR_PAGE;
      c = c < 0 ? 0 : limit;
    }
    int64_t a = c + n;
    if (a < 0) {
      err |= FP4MOE_ERR_PAGE;
      a = 0;
    }
    if (n > 0) tokens += n;
    if (a < c) back += pages((int32_t)c) - pages((int32_t)a);
    from[b] = (int32_t)c;
    to[b] = a > limit ? -1 : (int32_t)a;  // -1: no columns for it
  }
  int64_t all_tokens, all_back, all_need;
  int64_t at = block_sum(tokens, part, all_tokens), ab = block_sum(back, part, all_back);
  int64_t need = 0;
#pragma unroll
  for (int i = 0; i < KP_ITEMS; ++i) {
    const int b = b0 + i;
    if (i >= per || b >= B) break;
    const int32_t c = from[b];
    const int64_t n = fresh[i];
    first[b] = clamp32(at, p.rows);
    given[b] = clamp32(ab, INT32_MAX);
    if (n > 0) at += n;
    if (to[b] < 0 || (n > 0 && at > p.rows)) {  // takes nothing
      err |= FP4MOE_ERR_CAPACITY;
      to[b] = c;
      from[b] = ~c;
    } else if (to[b] < c) {
      ab += pages(c) - pages(to[b]);
    } else {
      need += pages(to[b]) - pages(c);
    }
  }
  int64_t an = block_sum(need, part, all_need);
  // ---- the stack
  int32_t F = *p.free_count;
  if (F < 0 || F > p.num_pages) {
    err |= FP4MOE_ERR_PAGE;
    F = F < 0 ? 0 : p.num_pages;
  }
  if (all_back > p.num_pages - F) err |= FP4MOE_ERR_PAGE;
  const int32_t P = clamp32(all_back, p.num_pages - F), top = F + P;
#pragma unroll
  for (int i = 0; i < KP_ITEMS; ++i) {
    const int b = b0 + i;
    if (i >= per || b >= B) break;
    taken[b] = clamp32(an, INT32_MAX);
    const int32_t c = from[b];
    if (c < 0 || to[b] <= c) continue;
    const int32_t k = pages(to[b]) - pages(c);
    if (k > 0 && an + k > top) {
      atomicMin(&first_refused, clamp32(an, INT32_MAX));
      err |= FP4MOE_ERR_CAPACITY;
      to[b] = c;
      from[b] = ~c;
    }
    an += k;
  }
  if (tid == 0) first[B] = clamp32(all_tokens, p.rows);
  if (err) atomicOr(&errors, err);
  __syncthreads();
  const int32_t Q = (int32_t)(all_need < first_refused ? all_need : first_refused);  // pages taken
  const int32_t total = first[B];
  // entry i of the pages given back, and entry v of the stack with them on top
  auto given_page = [&](int32_t i) {
    const int b = last_at_most(given, B, i);
    return p.table[(int64_t)b * p.columns + pages(to[b]) + (i - given[b])];
  };
  auto stack_page = [&](int32_t v) { return v < F ? p.free_pages[v] : given_page(v - F); };
  err = 0;
  const int step = (int)ctas * KP_THREADS, i0 = (int)rank * KP_THREADS + tid;
  // ---- tokens. Where there are more than threads, a thread takes four neighbours: one search, and mostly one page, for
  // them (512 sequences, 50000 tokens: 16.8 -> 14.2 us); else one each, so that the reads of all are under way at once.
  auto take = [&](int64_t t, int n, int32_t (&pos)[4], int32_t (&slot)[4]) {
    int b = t < total ? last_at_most(first, B, (int32_t)t) : 0;
    int32_t page = -1, page_at = -1, page_of = -1;  // the last page read: entry page_at of sequence page_of
#pragma unroll
    for (int i = 0; i < 4; ++i, ++t) {
      pos[i] = 0;
      slot[i] = -1;
      if (i >= n || t >= total) continue;
      while (t >= first[b + 1]) ++b;
      const int32_t c = from[b], k = (int32_t)t - first[b];
      if (c < 0) {
        pos[i] = clamp32((int64_t)~c + k, INT32_MAX);
        continue;
      }
      pos[i] = c + k;
      const int32_t j = (int32_t)p.page.div((uint32_t)pos[i]);
      if (j != page_at || b != page_of) {
        const int32_t old = pages(c);
        page = j < old ? p.table[(int64_t)b * p.columns + j] : stack_page(top - 1 - (taken[b] + j - old));
        page_at = j;
        page_of = b;
      }
      if (page >= 0 && page < p.num_pages) slot[i] = page * (int32_t)p.page.d + (pos[i] - j * (int32_t)p.page.d);
      else err |= FP4MOE_ERR_PAGE;
    }
  };
  if (p.rows > step) {
    for (int64_t t = (int64_t)i0 * 4; t < p.rows; t += (int64_t)step * 4) {
      int32_t pos[4], slot[4];
      const int n = (int)min((int64_t)4, p.rows - t);
      take(t, n, pos, slot);
      if (n == 4) {
        *reinterpret_cast<int4*>(p.position + t) = make_int4(pos[0], pos[1], pos[2], pos[3]);
        *reinterpret_cast<int4*>(p.slot + t) = make_int4(slot[0], slot[1], slot[2], slot[3]);
      } else {
        for (int i = 0; i < n; ++i) {
          p.position[t + i] = pos[i];
          p.slot[t + i] = slot[i];
        }
      }
    }
  } else if (i0 < p.rows) {
    int32_t pos[4], slot[4];
    take(i0, 1, pos, slot);
    p.position[i0] = pos[0];
    p.slot[i0] = slot[0];
  }
  // ---- pages taken, and those given back that stay on the stack
  for (int64_t k = i0; k < Q; k += step) {
    const int b = last_at_most(taken, B, (int32_t)k);
    p.table[(int64_t)b * p.columns + pages(from[b]) + ((int32_t)k - taken[b])] = stack_page(top - 1 - (int32_t)k);
  }
  for (int64_t i = i0; i < P - Q; i += step) p.free_pages[F + i] = given_page((int32_t)i);
  for (int b = i0; b <= B; b += step) p.q_offset[b] = first[b];
  if (err) atomicOr(&errors, err);
  // ---- outputs that may lie in an input's place
  cluster_sync();
  for (int b = i0; b < B; b += step) p.kv_len[b] = to[b];
  if (tid == 0) {
    if (rank == 0) *p.free_count_out = top - Q;
    if (errors) raise_error(p.err, errors);
  }
}

}  // namespace

fp4moe_status kv_plan_launch(int32_t num_seqs, int32_t page_size, int32_t num_pages, const int32_t* cached_len,
                             const int32_t* new_len, int32_t* page_table, int32_t table_columns, int32_t* free_pages,
                             const int32_t* free_count, int32_t* kv_len, int32_t* free_count_out, int32_t* q_offset,
                             int32_t rows, int32_t* position, int32_t* slot, uint32_t* err, cudaStream_t st) {
  KvPlanParams p{};
  p.B = num_seqs;
  p.columns = table_columns;
  p.num_pages = num_pages;
  p.rows = rows;
  p.page = FastDiv((uint32_t)page_size);
  p.cached = cached_len;
  p.fresh = new_len;
  p.table = page_table;
  p.free_pages = free_pages;
  p.free_count = free_count;
  p.kv_len = kv_len;
  p.free_count_out = free_count_out;
  p.q_offset = q_offset;
  p.position = position;
  p.slot = slot;
  p.err = err;
  const size_t smem = ((size_t)num_seqs * 5 + 1) * 4;
  static PerDevice done;
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return FP4MOE_CUDA_ERROR;
  if (done.get(dev, [] {
        return cudaFuncSetAttribute(kv_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    (FP4MOE_KV_MAX_SEQS * 5 + 1) * 4) == cudaSuccess
                   ? 1
                   : 0;
      }) <= 0)
    return FP4MOE_CUDA_ERROR;
  unsigned ctas = 1;
  while (ctas < KP_MAX_CLUSTER && (int64_t)ctas * KP_THREADS * 2 < rows) ctas *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(KP_THREADS);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ctas;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kv_plan_kernel, p) == cudaSuccess ? FP4MOE_OK : FP4MOE_CUDA_ERROR;
}

}  // namespace fp4moe
