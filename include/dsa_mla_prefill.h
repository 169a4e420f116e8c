/* Latent attention in its expanded form, for prompts: each head has keys and values of its
 * own, which the up-projection made from the latent rows, and the 64 rotary dims of the keys
 * are shared by all heads.  For a prompt this takes 2 * (192 + 128) operations a query, key
 * and head, where the absorbed form of dsa_sparse_attn.h takes 2 * (576 + 512).
 *
 * Request r has query rows cu_q[r] .. cu_q[r + 1] - 1 and key rows cu_kv[r] .. cu_kv[r + 1] - 1,
 * its context first and the queries' own tokens last: with q_len and kv_len their numbers,
 * query row i of the request sees its keys j with 0 <= j <= kv_len - q_len + i.  For each head
 *   k_j = (k_nope[j][h], k_rope[j]),  128 + 64 dims
 *   out[t][h] = sum_j softmax_j(softmax_scale * q[t][h].k_j) v[j][h],  128 dims
 *   lse[t][h] = natural-log sum-exp of the scaled scores (-inf, and out = 0, for a row that
 *               sees nothing)
 * Rows of q and out that belong to no request are neither used nor written.  Keys and values
 * that some query row of the request sees are finite; every other row may hold anything.  A
 * query that is not finite, or whose largest score is not in fp32, makes its own row NaN and no
 * other.
 *
 *   q        bf16 or fp16 (`type`), [n_tokens][h][192]: 128 dims against k_nope, then 64 against k_rope
 *   k_nope   the same type, [n_keys][h][128]
 *   k_rope   the same type, [n_keys][64], row pitch k_rope_ld
 *   v, out   the same type, [n_keys][h][128] and [n_tokens][h][128]
 *            each with a token pitch and a head pitch in elements, multiples of 8, below 2^38
 *            bytes, and 16-byte aligned; out overlaps no input
 *   cu_q     int32 [n_req + 1], ascending, within [0, n_tokens]; cu_kv likewise within
 *            [0, n_keys] (values outside are taken as the nearest bound)
 *   lse      fp32 [n_tokens][h] or NULL
 *   max_q_len, max_kv_len   what the requests' numbers of queries and keys are expected not to
 *            pass.  They choose how the work is split, not the result
 * The workspace needs no initialisation and holds the status word of the last call
 * (dsa_sparse_attn_read_status reads it).  Calls that share a workspace must not overlap on
 * the GPU.  The same inputs give the same bits.  On-chip waits are bounded: where one runs
 * out (after about 10 s without progress), the status gets DSA_STATUS_WAIT_TIMEOUT, and rows
 * may be missing or wrong.
 *
 * Numerics: products accumulate in fp32; scores, the running maximum and sums are fp32.  For
 * the product with the values, not for their sum, a softmax weight is rounded to the inputs'
 * type, the one that the matrix instruction takes beside them: by at most 2^-8 (bf16) or 2^-11
 * (fp16; 2^-25 of the row's largest weight where that is more) relative, so that out's error
 * beside its own rounding is at most about 2^-8 or 2^-11 of sum_j p_j |v_j|.
 *
 * The call is asynchronous on `stream` (a cudaStream_t, NULL = legacy default stream),
 * allocates nothing and can be captured in a CUDA graph.  It returns DSA_OK, or one of the
 * following with nothing enqueued:
 *   - DSA_ERR_INVALID_ARG: a bad size or parameter, a null or misaligned pointer;
 *   - DSA_ERR_UNSUPPORTED_SHAPE: h, n_req, n_tokens or n_keys not served;
 *   - DSA_ERR_WORKSPACE_TOO_SMALL;
 *   - DSA_ERR_UNSUPPORTED_DEVICE: not compute capability 10.3;
 *   - DSA_ERR_CUDA: a CUDA call failed, or the library was built such that the kernel did not
 *     get the 168 registers a thread that its roles redistribute.
 */
#ifndef DSA_MLA_PREFILL_H_
#define DSA_MLA_PREFILL_H_

#include <stddef.h>
#include <stdint.h>

#include "dsa_sparse_attn.h"

#ifdef __cplusplus
extern "C" {
#endif

#define DSA_MLA_BF16 0
#define DSA_MLA_FP16 1
#define DSA_MLA_MAX_HEADS 1024
#define DSA_MLA_MAX_REQ 8192
/* For tests of the failure path only: CTA 0 stops loading after a block of 128 keys and
 * waits for what nothing completes (about 1 s).  The call's status gets
 * DSA_STATUS_WAIT_TIMEOUT, and every role of the CTA stops, drains the tensor core and frees
 * its tensor memory.  Rows that the CTA shared are unspecified. */
#define DSA_MLA_FLAG_TEST_WAIT_TIMEOUT 2u

typedef struct dsa_mla_params {
  int32_t n_tokens;     /* rows of q and out, 0..2^30 */
  int32_t n_keys;       /* rows of k_nope, k_rope and v, 0..2^30 */
  int32_t n_req;        /* requests, 0..DSA_MLA_MAX_REQ */
  int32_t h;            /* heads, 1..DSA_MLA_MAX_HEADS */
  int32_t max_q_len;    /* >= 0 */
  int32_t max_kv_len;   /* >= 0 */
  int32_t type;         /* DSA_MLA_BF16 or DSA_MLA_FP16 */
  float softmax_scale;  /* finite; e.g. 1/sqrt(192) */
  uint32_t flags;       /* 0, or DSA_MLA_FLAG_TEST_WAIT_TIMEOUT */
} dsa_mla_params;

/* Fill `p` for the given shape: max_q_len = n_tokens, max_kv_len = n_keys, softmax_scale
 * 1/sqrt(192), type DSA_MLA_BF16, flags 0.  Returns DSA_OK or an error code as
 * dsa_mla_prefill_fwd would. */
int dsa_mla_params_init(dsa_mla_params* p, int32_t n_tokens, int32_t n_keys, int32_t n_req, int32_t h);

/* Bytes of device workspace the call needs for `p` on a GPU with `num_sms` SMs (num_sms <= 0:
 * the current device); 0 for invalid parameters.  It holds the status word, the list of tiles
 * and the partial results of tiles that several CTAs share. */
size_t dsa_mla_prefill_workspace_size(const dsa_mla_params* p, int num_sms);

int dsa_mla_prefill_fwd(const void* q, int64_t q_ld, int64_t q_hd, const void* k_nope, int64_t k_ld, int64_t k_hd,
                        const void* k_rope, int64_t k_rope_ld, const void* v, int64_t v_ld, int64_t v_hd,
                        const int32_t* cu_q, const int32_t* cu_kv, void* out, int64_t out_ld, int64_t out_hd,
                        float* lse, const dsa_mla_params* p, void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* DSA_MLA_PREFILL_H_ */
