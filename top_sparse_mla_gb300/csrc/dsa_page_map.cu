// Page map of one serving step (include/dsa_page_map.h): block tables, positions and cache
// slots of the new tokens from the requests' lengths, in one launch.
//
// Every CTA computes the two prefix sums over all requests (new tokens and new pages) in
// its own shared memory, so the CTAs need not wait for one another: the lengths are 8
// bytes a request and come from L2 after the first CTA.  Then the tokens, the new pages
// and the requests are spread over all threads of the grid, one each; a token or a page
// finds its request by a binary search in the prefix sums.  A page id is read from the
// table only where the request had it before the call and from the free list otherwise,
// so no thread reads an entry that another one writes.
//
// Bound by latency: three barriers, three dependent loads for a token that continues a page
// (the lengths, the lengths of its own request, the table) and some 64-bit divisions by the
// page size; one CTA has two barriers more for the status.  5.0 us for 16 requests of a token
// each and 7.0 for 1021 in a graph, 6.0 for 71 k tokens of 33 requests, whose 1.2 MB are 0.2 us
// of memory.

#include <cuda_runtime.h>
#include <stdint.h>

#include "dsa_page_map.h"

namespace dsa_map {

constexpr int THREADS = 512;
constexpr int WARPS = THREADS / 32;

struct Params {
  const int32_t *ctx, *fresh;
  int32_t* table;
  long long table_ld;
  const int32_t* free_pages;
  int32_t *cu, *kv_lens, *positions;
  int64_t* slots;
  int32_t *token_req, *info;
  int n_req, cols, n_free, page, n_tokens;
};

struct Request {
  long long ctx, kv;   // tokens before and after the call
  int old_pages, pages;   // pages before and after, as far as the table has columns
};

__device__ __forceinline__ Request request(const Params& P, int r) {
  Request q;
  q.ctx = max(P.ctx[r], 0);
  q.kv = q.ctx + max(P.fresh[r], 0);
  q.old_pages = (int)min((q.ctx + P.page - 1) / P.page, (long long)P.cols);
  q.pages = (int)min((q.kv + P.page - 1) / P.page, (long long)P.cols);
  return q;
}

// index of the last entry of s[0..n] that is <= v (s ascending, s[0] = 0 <= v < s[n]):
// among equal entries the last, which is the one that is not empty
__device__ __forceinline__ int find(const int* s, int n, int v) {
  int lo = 0, hi = n;   // s[lo] <= v < s[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (s[mid] <= v) lo = mid; else hi = mid;
  }
  return lo;
}

// The new tokens of all requests may be far more than n_tokens; sums stop at `top`
// (n_tokens + 1), and a sum that stops is associative like a plain one.
__device__ __forceinline__ int add_to(int a, int b, int top) {
  return (int)min((unsigned)a + (unsigned)b, (unsigned)top);
}

__global__ void __launch_bounds__(THREADS) page_map_kernel(const __grid_constant__ Params P) {
  extern __shared__ int smem[];
  __shared__ int s_tok_warp[WARPS], s_page_warp[WARPS];
  // a dependent launched with programmatic serialization may start now; it waits for this
  // kernel's completion before it reads
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  int* s_tok = smem;                   // [n_req + 1] exclusive prefix of the new tokens
  int* s_page = smem + P.n_req + 1;    // [n_req + 1] exclusive prefix of the new pages
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int n = P.n_req, top = P.n_tokens + 1;

  for (int r = tid; r < n; r += THREADS) {
    const Request q = request(P, r);
    s_tok[r] = (int)min(q.kv - q.ctx, (long long)top);
    s_page[r] = q.pages - q.old_pages;
  }
  __syncthreads();
  // each thread sums `per` consecutive requests (an odd number, so that the threads of a
  // warp read different banks), then a prefix over the threads, then its own requests again
  const int per = ((n + THREADS - 1) / THREADS) | 1;
  const int r0 = min(tid * per, n), r1 = min(r0 + per, n);
  int tok = 0, pg = 0;
  for (int r = r0; r < r1; ++r) {
    tok = add_to(tok, s_tok[r], top);
    pg += s_page[r];
  }
  int tok_in = tok, pg_in = pg;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int a = __shfl_up_sync(0xFFFFFFFFu, tok_in, o), b = __shfl_up_sync(0xFFFFFFFFu, pg_in, o);
    if (lane >= o) {
      tok_in = add_to(tok_in, a, top);
      pg_in += b;
    }
  }
  if (lane == 31) {
    s_tok_warp[w] = tok_in;
    s_page_warp[w] = pg_in;
  }
  __syncthreads();
  int tok_ex = __shfl_up_sync(0xFFFFFFFFu, tok_in, 1), pg_ex = __shfl_up_sync(0xFFFFFFFFu, pg_in, 1);
  if (lane == 0) tok_ex = pg_ex = 0;
  int all_tok = 0, all_page = 0;
#pragma unroll
  for (int u = 0; u < WARPS; ++u) {
    if (u < w) {
      tok_ex = add_to(tok_ex, s_tok_warp[u], top);
      pg_ex += s_page_warp[u];
    }
    all_tok = add_to(all_tok, s_tok_warp[u], top);
    all_page += s_page_warp[u];
  }
  for (int r = r0; r < r1; ++r) {
    const int a = s_tok[r], b = s_page[r];
    s_tok[r] = tok_ex;
    s_page[r] = pg_ex;
    tok_ex = add_to(tok_ex, a, top);
    pg_ex += b;
  }
  if (tid == 0) {
    s_tok[n] = all_tok;
    s_page[n] = all_page;
  }
  __syncthreads();

  const int step = gridDim.x * THREADS, first = blockIdx.x * THREADS + tid;
  int bad = 0;
  // new pages
  for (long long k = first; k < all_page; k += step) {
    const int i = (int)k;
    const int r = find(s_page, n, i);
    const int page = i < P.n_free ? P.free_pages[i] : -1;
    P.table[r * P.table_ld + request(P, r).old_pages + (i - s_page[r])] = max(page, -1);
  }
  // tokens
  const int live = min(all_tok, P.n_tokens);
  for (int t = first; t < P.n_tokens; t += step) {
    int r = -1, pos = 0;
    long long slot = -1;
    if (t < live) {
      r = find(s_tok, n, t);
      const Request q = request(P, r);
      const long long p = q.ctx + (t - s_tok[r]);
      const long long blk = p / P.page;
      pos = (int)min(p, 0x7FFFFFFFLL);
      if (blk < P.cols) {
        int page = -1;
        if (blk < q.old_pages) {
          page = P.table[r * P.table_ld + blk];
        } else {
          const int i = s_page[r] + (int)(blk - q.old_pages);
          if (i < P.n_free) page = P.free_pages[i];
        }
        if (page >= 0) slot = (long long)page * P.page + (int)(p - blk * P.page);
      }
    }
    P.positions[t] = pos;
    P.slots[t] = slot;
    if (P.token_req) P.token_req[t] = r;
  }
  // requests, with everything that the status says about them (one CTA, so that its word
  // is complete after one reduction and no other CTA clears it)
  for (int r = first; r <= n; r += step) P.cu[r] = min(s_tok[r], P.n_tokens);
  for (int r = first; r < n; r += step) P.kv_lens[r] = (int)min(request(P, r).kv, 0x7FFFFFFFLL);
  if (blockIdx.x == 0) {
    for (int r = tid; r < n; r += THREADS) {
      const Request q = request(P, r);
      if ((q.kv + P.page - 1) / P.page > P.cols || q.kv > 0x7FFFFFFFLL) bad |= DSA_STATUS_TABLE_FULL;
      // the page that the first new token continues, if the request has it already
      if (q.kv > q.ctx && q.ctx % P.page != 0 && q.ctx / P.page < P.cols &&
          P.table[r * P.table_ld + q.ctx / P.page] < 0)
        bad |= DSA_STATUS_OUT_OF_PAGES;
    }
    for (long long i = tid; i < min(all_page, P.n_free); i += THREADS)
      if (P.free_pages[i] < 0) bad |= DSA_STATUS_OUT_OF_PAGES;
    bad = __reduce_or_sync(0xFFFFFFFFu, bad);
    __syncthreads();   // s_tok_warp is read above
    if (lane == 0) s_tok_warp[w] = bad;
    __syncthreads();
    if (tid == 0) {
      for (int u = 0; u < WARPS; ++u) bad |= s_tok_warp[u];
      if (all_page > P.n_free) bad |= DSA_STATUS_OUT_OF_PAGES;
      if (all_tok > P.n_tokens) bad |= DSA_STATUS_TOKENS_FULL;
      P.info[0] = min(all_page, P.n_free);
      P.info[1] = bad;
    }
  }
}

static bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

}  // namespace dsa_map

extern "C" int dsa_page_map(const int32_t* ctx_lens, const int32_t* new_lens, int32_t n_req, int32_t* block_table,
                            int64_t table_ld, int32_t table_cols, const int32_t* free_pages, int32_t n_free,
                            int32_t page_size, int32_t n_tokens, int32_t* cu_new, int32_t* kv_lens,
                            int32_t* positions, int64_t* slots, int32_t* token_req, int32_t* info, void* stream) {
  using namespace dsa_map;
  if (n_req < 0 || n_tokens < 0 || n_tokens > (1 << 30) || page_size < 1 || n_free < 0) return DSA_ERR_INVALID_ARG;
  if (!cu_new || !info || !aligned(cu_new, 4) || !aligned(info, 4)) return DSA_ERR_INVALID_ARG;
  if (n_req > 0) {
    if (table_cols < 1 || table_ld < table_cols || (int64_t)n_req * table_cols >= (1LL << 31))
      return DSA_ERR_INVALID_ARG;
    if (!ctx_lens || !new_lens || !block_table || !kv_lens || !aligned(ctx_lens, 4) || !aligned(new_lens, 4) ||
        !aligned(block_table, 4) || !aligned(kv_lens, 4))
      return DSA_ERR_INVALID_ARG;
  }
  if (n_free > 0 && (!free_pages || !aligned(free_pages, 4))) return DSA_ERR_INVALID_ARG;
  if (n_tokens > 0 && (!positions || !slots || !aligned(positions, 4) || !aligned(slots, 8))) return DSA_ERR_INVALID_ARG;
  if (token_req && !aligned(token_req, 4)) return DSA_ERR_INVALID_ARG;
  if (n_req > DSA_PAGE_MAP_MAX_REQ) return DSA_ERR_UNSUPPORTED_SHAPE;
  int dev = 0, major = 0, minor = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return DSA_ERR_CUDA;
  cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev);
  cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev);
  if (major != 10 || minor != 3) return DSA_ERR_UNSUPPORTED_DEVICE;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return DSA_ERR_CUDA;
  Params P;
  P.ctx = ctx_lens;
  P.fresh = new_lens;
  P.table = block_table;
  P.table_ld = (long long)table_ld;
  P.free_pages = free_pages;
  P.cu = cu_new;
  P.kv_lens = kv_lens;
  P.positions = positions;
  P.slots = slots;
  P.token_req = token_req;
  P.info = info;
  P.n_req = n_req;
  P.cols = n_req > 0 ? table_cols : 1;
  P.n_free = n_free;
  P.page = page_size;
  P.n_tokens = n_tokens;
  const size_t smem = (size_t)2 * (n_req + 1) * sizeof(int);
  if (smem > 40 * 1024) {   // 48 KB are for dynamic and static shared memory together, and the latter is below 8 KB
    // raised on every call that needs it: it costs less than a microsecond, and only
    // batches of more than 5119 requests come here
    if (cudaFuncSetAttribute(page_map_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)(2 * (DSA_PAGE_MAP_MAX_REQ + 1) * sizeof(int))) != cudaSuccess)
      return DSA_ERR_CUDA;
  }
  const int most = n_tokens > n_req + 1 ? n_tokens : n_req + 1;
  int grid = (most + THREADS - 1) / THREADS;
  if (grid > sms) grid = sms;
  page_map_kernel<<<grid, THREADS, smem, (cudaStream_t)stream>>>(P);
  return cudaGetLastError() == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}
