/* Latent rows read back from the cache: the fp8_ds_mla rows (dsa_kv_insert.h) that a batch
 * of requests' block tables name, dequantised into dense bf16 rows.  This is what the
 * up-projection in front of dsa_mla_prefill_fwd reads for the part of a context that the
 * cache holds already.
 *
 * Request r's rows of the output are cu_rows[r] .. cu_rows[r + 1] - 1.  Row cu_rows[r] + i,
 * for i < lens[r] (all of them where lens is NULL), becomes
 *   - values 0..511: e4m3 code * scale of its block of 128, rounded to fp32 and then to bf16;
 *   - values 512..575: the 64 rotary values, as they are stored;
 * of pool row block_table[r][i / page_size] * page_size + i % page_size.  A row whose table
 * entry is negative, past table_cols or points past n_rows becomes 0, and
 * DSA_STATUS_SLOT_OUT_OF_RANGE is OR-ed into *status.  Rows of no request, those from lens[r]
 * on and the columns from 576 on stay as they were.
 *
 *   pool         uint8 [n_rows][656], 16-byte aligned; n_rows >= 0
 *   block_table  int32 [n_req][table_cols], row pitch table_ld
 *   cu_rows      int32 [n_req + 1], ascending, within [0, n_out] (values outside are taken as
 *                the nearest bound)
 *   lens         int32 [n_req] or NULL
 *   out          bf16 [n_out][ld], ld >= 576, ld % 8 == 0, 16-byte aligned; overlaps no input
 *   status       uint32 (device, 4-byte aligned) or NULL; the caller clears it
 *   n_req >= 0, n_out >= 0, table_cols >= 0, page_size >= 1
 * The call is asynchronous on `stream` (a cudaStream_t, NULL = legacy default stream),
 * allocates nothing, launches one kernel, and can be captured in a CUDA graph.  It returns
 * DSA_OK, or one of the following with nothing enqueued:
 *   - DSA_ERR_INVALID_ARG: a bad size, a null or misaligned pointer;
 *   - DSA_ERR_UNSUPPORTED_DEVICE: not compute capability 10.3;
 *   - DSA_ERR_CUDA.
 */
#ifndef DSA_KV_GATHER_H_
#define DSA_KV_GATHER_H_

#include <stdint.h>

#include "dsa_kv_insert.h"
#include "dsa_sparse_attn.h"

#ifdef __cplusplus
extern "C" {
#endif

int dsa_kv_gather(const void* pool, int64_t n_rows, const int32_t* block_table, int64_t table_ld, int32_t table_cols,
                  int32_t page_size, const int32_t* cu_rows, const int32_t* lens, int32_t n_req, void* out,
                  int64_t ld, int32_t n_out, uint32_t* status, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* DSA_KV_GATHER_H_ */
