/* Page map of one serving step: block tables, positions and cache slots of the new tokens,
 * built on the GPU from the requests' lengths.  It produces the `positions` and `slots`
 * that dsa_kv_insert reads, and the `slots`, `block_table`, `cu_new` and `kv_lens` that
 * dsa_kv8_insert and dsa_kv8_attn_fwd read.
 *
 * A paged cache holds request r's token at position p in row p % page_size of page
 * block_table[r][p / page_size].  With ctx_lens[r] tokens in the cache and new_lens[r]
 * tokens to add (a negative length counts as 0), the call computes
 *   - cu_new[r] = sum of new_lens[s] over s < r, for r = 0..n_req: request r's new tokens
 *     are rows cu_new[r] .. cu_new[r + 1] - 1 of the batch;
 *   - kv_lens[r] = ctx_lens[r] + new_lens[r];
 *   - the pages that the new tokens need beyond the ceil(ctx_lens[r] / page_size) that
 *     the request has: taken from free_pages[0], [1], ... in request order and written to
 *     block_table[r]; no other entry of the table is written;
 *   - for each new token: positions[t] = ctx_lens[r] + (t - cu_new[r]),
 *     slots[t] = page * page_size + positions[t] % page_size, token_req[t] = r;
 *   - for the rows t of a padded batch behind the last new token: positions[t] = 0,
 *     slots[t] = -1 (skipped by both inserts), token_req[t] = -1;
 *   - info[0] = pages taken from the list, info[1] = DSA_STATUS_* bits.
 * What does not fit is reported in info[1], and every other value stays as described:
 *   - DSA_STATUS_OUT_OF_PAGES: a page was needed past the end of the list (or its entry
 *     in the list, or the request's own table entry, was negative): the table entry is
 *     -1 where it came from the list, and the tokens in it get slot -1;
 *   - DSA_STATUS_TABLE_FULL: a request needs more than table_cols pages (or its length
 *     passes 2^31 - 1, which kv_lens then holds): tokens past the last column get slot -1;
 *   - DSA_STATUS_TOKENS_FULL: the new tokens are more than n_tokens: the rows past
 *     n_tokens are not mapped, and cu_new stops at n_tokens.
 *
 * Arguments (device pointers, owned by the caller; outputs overlap neither each other nor
 * the inputs):
 *   ctx_lens, new_lens  int32 [n_req]
 *   block_table         int32 [n_req][table_ld], in and out; table_ld >= table_cols >= 1
 *   free_pages          int32 [n_free] (may be NULL when n_free == 0)
 *   cu_new              int32 [n_req + 1]
 *   kv_lens             int32 [n_req]
 *   positions           int32 [n_tokens]
 *   slots               int64 [n_tokens]
 *   token_req           int32 [n_tokens] or NULL
 *   info                int32 [2]
 *   0 <= n_req <= DSA_PAGE_MAP_MAX_REQ, 0 <= n_tokens <= 2^30, page_size >= 1, n_free >= 0,
 *   n_req * table_cols < 2^31.
 * With n_tokens == 0, positions, slots and token_req may be NULL.  With n_req == 0 the
 * other arrays by request may be NULL; the padding rows, cu_new[0] and info are written.
 * The call is asynchronous on `stream` (a cudaStream_t, NULL = legacy default stream),
 * allocates nothing, launches one kernel, and can be captured in a CUDA graph.  It returns
 * DSA_OK, or one of the following with nothing enqueued:
 *   - DSA_ERR_INVALID_ARG: a bad size, a null or misaligned pointer;
 *   - DSA_ERR_UNSUPPORTED_SHAPE: n_req above DSA_PAGE_MAP_MAX_REQ;
 *   - DSA_ERR_UNSUPPORTED_DEVICE: not compute capability 10.3;
 *   - DSA_ERR_CUDA.
 */
#ifndef DSA_PAGE_MAP_H_
#define DSA_PAGE_MAP_H_

#include <stdint.h>

#include "dsa_sparse_attn.h"

#ifdef __cplusplus
extern "C" {
#endif

#define DSA_PAGE_MAP_MAX_REQ 8192   /* the requests' prefix sums are held in shared memory */
#define DSA_STATUS_OUT_OF_PAGES 8u  /* a new token's page was missing */
#define DSA_STATUS_TABLE_FULL 16u   /* a request needs more pages than the table has columns */
#define DSA_STATUS_TOKENS_FULL 32u  /* more new tokens than n_tokens */

int dsa_page_map(const int32_t* ctx_lens, const int32_t* new_lens, int32_t n_req, int32_t* block_table,
                 int64_t table_ld, int32_t table_cols, const int32_t* free_pages, int32_t n_free,
                 int32_t page_size, int32_t n_tokens, int32_t* cu_new, int32_t* kv_lens, int32_t* positions,
                 int64_t* slots, int32_t* token_req, int32_t* info, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* DSA_PAGE_MAP_H_ */
