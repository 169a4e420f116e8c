/* Attention over a paged key/value cache held in 8 bits, and the insert that fills it.
 *
 * Cache.  Two pools (keys and values) of n_pages pages; a page holds page_size tokens of
 * every KV head, E4M3 codes with one fp32 scale per page and head:
 *   k_pool, v_pool    uint8 [n_pages][h_kv][page_size][d]   16-byte aligned
 *   k_scale, v_scale  fp32  [n_pages][h_kv]
 * The value of a code is e4m3 * scale.  A request's token at position p is row
 * p % page_size of page block_table[r][p / page_size] (see dsa_page_map.h, which builds
 * the tables and the slots page * page_size + p % page_size).
 *   d is 64 or 128; page_size is 16, 32, 64 or 128; 1 <= h_kv <= DSA_KV8_MAX_HEADS;
 *   n_pages * h_kv * page_size < 2^32 - 1.
 *
 * ---- dsa_kv8_insert: quantise new tokens' keys and values into their pages.
 * Token i of the batch goes to row slots[i] % page_size of page slots[i] / page_size;
 * slots[i] < 0 skips it (padding).  The new tokens of one page are a run: consecutive
 * tokens of the batch with consecutive slots, as dsa_page_map numbers them.  Let the run
 * begin at row o0 of its page, and let amax be the largest magnitude among the run's
 * finite values of one head (0 if there is none).  For each page and head, keys and values
 * apart:
 *   - s = the least power of two with amax <= 448 s, within [2^-64, 2^64];
 *   - with o0 > 0 the rows before o0 are tokens that the page holds already: s is raised
 *     to the page's scale if that is larger, and where s is larger than the page's scale
 *     those rows' codes become the E4M3 values nearest to code * (old scale / s);
 *   - the new rows' codes are the E4M3 values nearest to x * (1 / s) (ties to even,
 *     saturating), and the page's scale becomes s.  Scales that are powers of two make
 *     every product here exact, so a value's code does not depend on how its page was
 *     filled, but for values below 2^-6 s that were rounded at an earlier scale.
 * With o0 == 0 the page's old contents are forgotten.  Rows behind the run and other
 * pages are left as they were.  Non-finite inputs: an infinity saturates, a NaN gives the
 * E4M3 NaN code, and neither changes the scale.  If two runs of one call share a page, or
 * a slot occurs twice, that page's codes and scale are unspecified (nothing else is).
 *   k, v    bf16 or fp16 (`type`) [n_tokens][h_kv][d]: token pitch ld and head pitch hd in
 *           elements, both multiples of 8, hd >= d unless h_kv == 1; 16-byte aligned
 *   slots   int64 [n_tokens]
 *   status  uint32 (device, 4-byte aligned) or NULL: a slot >= n_pages * page_size is
 *           skipped, and DSA_STATUS_SLOT_OUT_OF_RANGE is OR-ed into *status (the caller
 *           clears it)
 * One kernel; the new tokens are read once.
 *
 * ---- dsa_kv8_attn_fwd: attention of a ragged batch of queries over the cache.
 * Request r has query rows cu_q[r] .. cu_q[r + 1] - 1 and kv_lens[r] tokens in the cache,
 * the queries' own among them: query row i of the request is at position
 * p = kv_lens[r] - q_len + i and sees the positions j with 0 <= j <= p and, with
 * window > 0, j > p - window.  Query head h reads KV head h / (h_q / h_kv):
 *   out[t][h] = sum_j softmax_j(softmax_scale * q[t][h].k_j) v_j
 *   lse[t][h] = natural-log sum-exp of the scaled scores (-inf, and out = 0, for a row
 *               that sees nothing)
 * A query that is not finite makes its own row NaN, or, where every score that it sees is
 * -infinity, 0 with an lse of -inf; no other row.
 * A table entry that is negative or >= n_pages holds nothing: its positions are not seen.
 * Rows of q and out that belong to no request are neither read nor written.  Codes of
 * rows that some query row of the request sees are finite, with positive finite scales
 * (value scales outside [2^-64, 2^64] count as the nearer bound); everything else in the
 * pools and tables may hold anything (pages past a request's length, rows past it inside
 * its last page, pages before the first row's window).
 *   q, out       bf16 or fp16 (`type`), [n_tokens][h_q][d]: token pitch and head pitch in
 *                elements, both multiples of 8; 16-byte aligned; out overlaps no input
 *   block_table  int32 [n_req][table_cols], row pitch table_ld
 *   cu_q         int32 [n_req + 1], ascending, within [0, n_tokens] (values outside are
 *                taken as the nearest bound)
 *   kv_lens      int32 [n_req] (values outside [0, table_cols * page_size] are taken as the
 *                nearest bound, the queries' positions with them)
 *   lse          fp32 [n_tokens][h_q] or NULL
 *   max_q_len    no request has more query rows (a request that does is skipped, its rows
 *                unwritten, and the call's status gets DSA_STATUS_QUERY_TOO_LONG); it
 *                selects the kernels that the call launches
 * The workspace needs no initialisation and holds the status word of the last call
 * (dsa_sparse_attn_read_status reads it).  Calls that share a workspace must not overlap
 * on the GPU.  Results do not depend on the other requests' order of completion: the same
 * inputs give the same bits.  On-chip waits are bounded: where one runs out (after about 10 s),
 * the status gets DSA_STATUS_WAIT_TIMEOUT, and rows may be missing or wrong.
 *
 * Numerics: E4M3 codes are exact in fp16, and so are the queries after each row's scaling
 * by a power of two, down to 2^-22 (fp16) or 2^-25 (bf16) of the row's largest magnitude;
 * smaller ones are rounded, by at most 2^-32 of the largest.  Products accumulate in fp32;
 * scores, the running maximum and sums are fp32.  For the product with the values, not for
 * their sum, the softmax weight p_j of a token times its page's value scale is rounded to
 * fp16: by 2^-11 relative, or by 2^-25 of the largest p_j * v_scale_j of the row where that
 * is more.  So out's error beside its own rounding is at most 2^-11 sum_j p_j |v_j| and
 * 2^-25 max_j(p_j * v_scale_j) sum_j |code_j|: a page whose value scale is far below another's
 * that the row sees counts with fewer bits, in dims where the other page's values are small.
 *
 * Both calls are asynchronous on `stream` (a cudaStream_t, NULL = legacy default stream),
 * allocate nothing and can be captured in a CUDA graph.  They return DSA_OK, or one of the
 * following with nothing enqueued:
 *   - DSA_ERR_INVALID_ARG: a bad size or parameter, a null or misaligned pointer;
 *   - DSA_ERR_UNSUPPORTED_SHAPE: d, page_size, h_kv, h_q / h_kv, n_req or a product of sizes
 *     not served (attention: n_tokens * h_q / h_kv < 2^31; a window above 2^30 only with
 *     table_cols * page_size <= 2^30);
 *   - DSA_ERR_WORKSPACE_TOO_SMALL (attention);
 *   - DSA_ERR_UNSUPPORTED_DEVICE: not compute capability 10.3;
 *   - DSA_ERR_CUDA: a CUDA call failed, or the library was built such that the kernel for
 *     many query rows did not get the 128 registers a thread that its roles redistribute
 *     (with another compiler, or flags for debugging).
 */
#ifndef DSA_KV8_H_
#define DSA_KV8_H_

#include <stddef.h>
#include <stdint.h>

#include "dsa_kv_insert.h"
#include "dsa_sparse_attn.h"

#ifdef __cplusplus
extern "C" {
#endif

#define DSA_KV8_BF16 0
#define DSA_KV8_FP16 1
#define DSA_KV8_MAX_HEADS 1024          /* KV heads */
#define DSA_KV8_MAX_GROUP 128           /* query heads per KV head */
#define DSA_KV8_MAX_REQ 8192            /* requests of one attention call */
/* For tests of the failure path only: CTA 0 of the kernel that serves requests of many query
 * rows (more than 32 with their heads, by KV head) stops copying after three blocks of 128
 * cached tokens and waits for what nothing completes.  That wait runs out (about 1 s), the
 * call's status gets DSA_STATUS_WAIT_TIMEOUT, and every role of the CTA stops, drains the
 * tensor core and frees its tensor memory.  Rows that the CTA did not finish are unwritten
 * or, where a cluster shares them, unspecified; the others are complete. */
#define DSA_KV8_FLAG_TEST_WAIT_TIMEOUT 2u
#define DSA_STATUS_QUERY_TOO_LONG 64u   /* a request had more than max_q_len query rows */

int dsa_kv8_insert(const void* k, int64_t k_ld, int64_t k_hd, const void* v, int64_t v_ld, int64_t v_hd,
                   const int64_t* slots, int32_t n_tokens, int32_t type, void* k_pool, void* v_pool,
                   float* k_scale, float* v_scale, int32_t n_pages, int32_t h_kv, int32_t page_size, int32_t d,
                   uint32_t* status, void* stream);

typedef struct dsa_kv8_params {
  int32_t n_tokens;     /* rows of q and out (>= 0) */
  int32_t n_req;        /* requests, 0..DSA_KV8_MAX_REQ */
  int32_t h_q;          /* query heads, a multiple of h_kv */
  int32_t h_kv;         /* KV heads */
  int32_t d;            /* head dimension, 64 or 128 */
  int32_t page_size;    /* 16, 32, 64 or 128 */
  int32_t n_pages;      /* pages in each pool */
  int32_t table_cols;   /* columns of the block table */
  int32_t max_q_len;    /* >= 0 */
  int32_t window;       /* 0: none */
  int32_t type;         /* DSA_KV8_BF16 or DSA_KV8_FP16 */
  float softmax_scale;  /* finite; e.g. 1/sqrt(d) */
  uint32_t flags;       /* 0, or DSA_KV8_FLAG_TEST_WAIT_TIMEOUT */
} dsa_kv8_params;

/* Fill `p` for the given shape: max_q_len = n_tokens, window 0, softmax_scale 1/sqrt(d),
 * type DSA_KV8_BF16, flags 0.  Returns DSA_OK or an error code as dsa_kv8_attn_fwd would. */
int dsa_kv8_params_init(dsa_kv8_params* p, int32_t n_tokens, int32_t n_req, int32_t h_q, int32_t h_kv, int32_t d,
                        int32_t page_size, int32_t n_pages, int32_t table_cols);

/* Bytes of device workspace the attention needs for `p` on a GPU with `num_sms` SMs
 * (num_sms <= 0: the current device); 0 for invalid parameters.  It holds the status
 * word, the work lists, and the partial results of requests that several CTAs share. */
size_t dsa_kv8_attn_workspace_size(const dsa_kv8_params* p, int num_sms);

int dsa_kv8_attn_fwd(const void* q, int64_t q_ld, int64_t q_hd, const void* k_pool, const void* v_pool,
                     const float* k_scale, const float* v_scale, const int32_t* block_table, int64_t table_ld,
                     const int32_t* cu_q, const int32_t* kv_lens, void* out, int64_t out_ld, int64_t out_hd,
                     float* lse, const dsa_kv8_params* p, void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* DSA_KV8_H_ */
