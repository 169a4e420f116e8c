/* Attention over the paged 8-bit cache for a batch whose requests share prefixes: a system
 * prompt, or several answers to one prompt.  The result is that of dsa_kv8_attn_fwd (dsa_kv8.h,
 * which defines the cache, the arguments and the numerics); the pages that a group of requests
 * shares are read once for the queries of all of them.
 *
 * Group g has the requests cu_groups[g] .. cu_groups[g + 1] - 1, whose block tables name the
 * same pages for the whole pages among their first prefix_lens[g] tokens.  The call takes what
 * the group shares from the table of one of its requests that has queries, as far as every
 * query of the group sees it: the least of prefix_lens[g] and of kv_len - q_len + 1 over the
 * group's requests with queries, in whole pages, and at most 2^31 - 1024 - n_tokens tokens.  So
 * a prefix length may be too large by what is not seen, but not by pages that differ, and it is
 * right, if slower, to give less.
 * Requests outside every group share nothing.
 *
 *   cu_groups    int32 [n_groups + 1], ascending, within [0, n_req] (values outside are taken
 *                as the nearest bound)
 *   prefix_lens  int32 [n_groups] (negative: 0)
 *   n_groups     0 (neither array is read) to DSA_KV8_MAX_GROUPS; n_req + n_groups <= DSA_KV8_MAX_REQ
 *   window has to be 0
 * What the call saves is reading, (n - 1) times a prefix for a group of n requests; it costs
 * two kernels more and a pass over O in fp32.  On a GB300 it is the faster one for groups of
 * eight and more from about 250 MB of codes saved in a call on (16 requests behind 8 k tokens
 * or 64 behind 2 k, 8 KV heads of 128), for groups of four from about 1 GB; for pairs, for
 * prompts of some hundred tokens and for chunks of 128 queries and more, dsa_kv8_attn_fwd is.
 * All other arguments, the status word of the workspace, what is left unwritten, and the rules
 * for streams and graphs are those of dsa_kv8_attn_fwd.  Beside its error, O and the sums of
 * the two parts of a row, the shared tokens and its own, are joined in fp32.
 *
 * The call returns DSA_OK or an error as dsa_kv8_attn_fwd does, with nothing enqueued;
 * DSA_ERR_UNSUPPORTED_SHAPE also for a window or too many groups, DSA_ERR_INVALID_ARG also for
 * n_groups < 0 and for null or misaligned arrays of the groups. */
#ifndef DSA_KV8_PREFIX_H_
#define DSA_KV8_PREFIX_H_

#include <stddef.h>
#include <stdint.h>

#include "dsa_kv8.h"

#ifdef __cplusplus
extern "C" {
#endif

#define DSA_KV8_MAX_GROUPS 4096

/* Bytes of device workspace for `p` and n_groups on a GPU with `num_sms` SMs (num_sms <= 0: the
 * current device); 0 for invalid parameters. */
size_t dsa_kv8_prefix_workspace_size(const dsa_kv8_params* p, int32_t n_groups, int num_sms);

int dsa_kv8_prefix_attn_fwd(const void* q, int64_t q_ld, int64_t q_hd, const void* k_pool, const void* v_pool,
                            const float* k_scale, const float* v_scale, const int32_t* block_table, int64_t table_ld,
                            const int32_t* cu_q, const int32_t* kv_lens, const int32_t* cu_groups,
                            const int32_t* prefix_lens, int32_t n_groups, void* out, int64_t out_ld, int64_t out_hd,
                            float* lse, const dsa_kv8_params* p, void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* DSA_KV8_PREFIX_H_ */
