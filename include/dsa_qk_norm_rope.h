/* Queries and keys of an attention layer made ready: RMS norm of each head and rotary
 * position embedding, in one pass over both.  Its keys are what dsa_kv8_insert quantises,
 * its queries what dsa_kv8_attn_fwd and dsa_kv8_prefix_attn_fwd read; with the rotary dims
 * at a head's end and without a norm, it makes the queries and rotary keys of
 * dsa_mla_prefill_fwd.
 *
 * For every token t, every one of the h_q heads of q and the h_k heads of k, x the head's d
 * values:
 *   - y = x / sqrt(mean(x^2) + rms_eps) * w, with w the d weights of q or of k; without
 *     weights (NULL) y = x;
 *   - the rotary_dim values from rotary_start on are taken in pairs (a_i, b_i), i = 0 ..
 *     rotary_dim / 2 - 1: values i and i + rotary_dim / 2 of them, or, with
 *     DSA_QK_FLAG_INTERLEAVED, 2i and 2i + 1.  Each pair turns by positions[t] *
 *     rope_base^(-2i / rotary_dim): (a cos - b sin, a sin + b cos); the other values stay y;
 *   - the result is rounded once to the inputs' type.
 * Statistics, weights' products and rotations are fp32 (squares of magnitudes above 2^63
 * overflow); an angle's fraction of a turn is exact to 2^-24 at every position.
 *
 *   q, k          bf16 or fp16 (`type`), [n_tokens][h][d]: token pitch ld and head pitch hd in
 *                 elements, multiples of 8; 16-byte aligned.  h_k may be 0 (k unused)
 *   q_w, k_w      the same type, [d], 16-byte aligned, or NULL
 *   positions     int32 [n_tokens] (may be negative)
 *   q_out, k_out  as q and k, with pitches of their own; either may be its input itself (the
 *                 same address and pitches), otherwise outputs overlap nothing
 *   d             a multiple of 16, 64..256; rotary_dim a multiple of 16, 0..d; rotary_start a
 *                 multiple of 8, rotary_start + rotary_dim <= d
 *   n_tokens >= 0, h_q >= 1, h_k >= 0, h_q + h_k <= DSA_QK_MAX_HEADS, rms_eps >= 0, rope_base > 0
 * The call is asynchronous on `stream` (a cudaStream_t, NULL = legacy default stream),
 * allocates nothing, launches one kernel, and can be captured in a CUDA graph.  It returns
 * DSA_OK, or one of the following with nothing enqueued:
 *   - DSA_ERR_INVALID_ARG: a bad size or parameter, a null or misaligned pointer;
 *   - DSA_ERR_UNSUPPORTED_SHAPE: d, rotary_dim, rotary_start or the heads not served;
 *   - DSA_ERR_UNSUPPORTED_DEVICE: not compute capability 10.3;
 *   - DSA_ERR_CUDA.
 */
#ifndef DSA_QK_NORM_ROPE_H_
#define DSA_QK_NORM_ROPE_H_

#include <stdint.h>

#include "dsa_sparse_attn.h"

#ifdef __cplusplus
extern "C" {
#endif

#define DSA_QK_BF16 0
#define DSA_QK_FP16 1
#define DSA_QK_FLAG_INTERLEAVED 1u   /* rotary pairs are neighbours */
#define DSA_QK_MAX_HEADS 4096        /* heads of queries and keys together */

typedef struct dsa_qk_params {
  int32_t n_tokens;
  int32_t h_q;
  int32_t h_k;
  int32_t d;
  int32_t rotary_dim;
  int32_t rotary_start;
  int32_t type;       /* DSA_QK_BF16 or DSA_QK_FP16 */
  uint32_t flags;
  float rms_eps;
  float rope_base;
} dsa_qk_params;

/* Fill `p` for the given shape: rotary_dim = d, rotary_start 0, type DSA_QK_BF16, flags 0,
 * rms_eps 1e-6, rope_base 10000.  Returns DSA_OK or an error code as dsa_qk_norm_rope would. */
int dsa_qk_params_init(dsa_qk_params* p, int32_t n_tokens, int32_t h_q, int32_t h_k, int32_t d);

int dsa_qk_norm_rope(const void* q, int64_t q_ld, int64_t q_hd, const void* k, int64_t k_ld, int64_t k_hd,
                     const int32_t* positions, const void* q_w, const void* k_w, void* q_out, int64_t q_out_ld,
                     int64_t q_out_hd, void* k_out, int64_t k_out_ld, int64_t k_out_hd, const dsa_qk_params* p,
                     void* stream);

#ifdef __cplusplus
}
#endif

#endif /* DSA_QK_NORM_ROPE_H_ */
