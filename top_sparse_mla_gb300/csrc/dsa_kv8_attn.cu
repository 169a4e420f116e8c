// Attention over the paged 8-bit cache (include/dsa_kv8.h).
//
// A call is a one-CTA plan kernel and the attention kernels as its programmatic dependents.
// They read the call's inputs before the plan is done: what wrote those precedes the plan
// kernel, which waits for it.
//
// Rows.  The query rows of one request and KV head are its q_len queries times the
// h_q / h_kv heads that share the KV head: row = query * group + head of the group, so
// every cached token is read once for all of them.  Requests with at most 8 * NT rows
// (decode, drafted tokens) go to rows_kernel below; the others are cut into tiles.
//
// What bounds rows_kernel: memory for 8 rows (64 requests of up to 32k tokens, 64/8 heads of
// 128: 2.04 GB in 308 us, 6.6 TB/s, 0.97 of a copy's rate); the latency of a step for 16 (48
// requests of up to 8k, 4 queries, 90 us, 0.67) and 32 rows, whose registers leave 12 and 8
// warps on an SM; ramp and join, about 10 us, for one request of 32k (20.1 us, floor 10).
//
// Scales.  With S = q . code_k summed in fp32 and x = S * k_scale * softmax_scale * log2 e,
// the kernels take t = x + log2(v_scale) and w = 2^(t - m), m a running maximum of t.  Then
// O = sum w * code_v is the weighted sum with every page's value scale in it, and
// l = sum w / v_scale is the softmax's sum (see SMALL_SCALE): w is at most 2^8 (the maximum may
// lag by 8), whatever the scales' magnitudes, so that it fits fp16.
//
// That w is rounded to fp16 for its product (2^-11, and 2^-25 of a row's largest) is a choice: a
// second product with what the rounding left would double that contraction, half of the work, and
// the result's own rounding hides it.  Against 64 bits bf16 outputs are off by 0.0017 of their norm,
// with w in fp32 by the same; fp16 ones under a window of 640 by 0.00023, in fp32 by 0.00021.

#include "device.cuh"
#include "dsa_kv8_rows.cuh"

namespace dsa_kv8 {

static void set_clusters(Params& P, const dsa_kv8_params* p, int max_tiles, int sms) {
  // cached tokens that a tile's rows may see
  const long long seen = P.window > 0 ? (long long)P.window + TILE_ROWS / P.group + 1 + STEP : P.cap;
  const long long pairs = (long long)max_tiles * p->h_kv;
  P.cluster = P.has_tiles && 2 * pairs <= sms ? cluster_size(p->d, pairs, (int)((min(seen, (long long)P.cap) + 127) / 128)) : 0;
  P.n_ctas = P.cluster ? (int)pairs * P.cluster : sms;
}

template <int D>
static int launch_all(const dsa_kv8_params* p, const Params& P, bool wide, cudaStream_t st) {
  const int nt = row_tiles(p);
  const int rc = nt == 1 ? launch_rows<D, 1, false>(P, wide, st) : nt == 2 ? launch_rows<D, 2, false>(P, wide, st) : launch_rows<D, 4, false>(P, wide, st);
  if (rc != DSA_OK) return rc;
  return has_tiles(p) ? launch_tiles(D, P, st) : DSA_OK;
}

}  // namespace dsa_kv8

extern "C" {

int dsa_kv8_params_init(dsa_kv8_params* p, int32_t n_tokens, int32_t n_req, int32_t h_q, int32_t h_kv, int32_t d,
                        int32_t page_size, int32_t n_pages, int32_t table_cols) {
  if (!p) return DSA_ERR_INVALID_ARG;
  p->n_tokens = n_tokens;
  p->n_req = n_req;
  p->h_q = h_q;
  p->h_kv = h_kv;
  p->d = d;
  p->page_size = page_size;
  p->n_pages = n_pages;
  p->table_cols = table_cols;
  p->max_q_len = n_tokens;
  p->window = 0;
  p->type = DSA_KV8_BF16;
  p->softmax_scale = d > 0 ? (float)(1.0 / sqrt((double)d)) : 1.0f;
  p->flags = 0;
  return dsa_kv8::check(p);
}

size_t dsa_kv8_attn_workspace_size(const dsa_kv8_params* p, int num_sms) {
  if (dsa_kv8::check(p) != DSA_OK) return 0;
  if (num_sms <= 0 && dsa::current_sms(&num_sms) != DSA_OK) return 0;
  return dsa_kv8::layout(p, num_sms).bytes;
}

int dsa_kv8_attn_fwd(const void* q, int64_t q_ld, int64_t q_hd, const void* k_pool, const void* v_pool,
                     const float* k_scale, const float* v_scale, const int32_t* block_table, int64_t table_ld,
                     const int32_t* cu_q, const int32_t* kv_lens, void* out, int64_t out_ld, int64_t out_hd, float* lse,
                     const dsa_kv8_params* p, void* workspace, size_t workspace_bytes, void* stream) {
  using namespace dsa_kv8;
  const int rc = check(p);
  if (rc != DSA_OK) return rc;
  const Call c{q, q_ld, q_hd, k_pool, v_pool, k_scale, v_scale, block_table, table_ld, cu_q, kv_lens, out, out_ld, out_hd, lse, workspace};
  if (bad_call(c, p)) return DSA_ERR_INVALID_ARG;
  int sms = 0;
  const int rc0 = dsa::gb300_sms(&sms);
  if (rc0 != DSA_OK) return rc0;
  const Layout L = layout(p, sms);
  if (workspace_bytes < L.bytes) return DSA_ERR_WORKSPACE_TOO_SMALL;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  cudaStream_t st = (cudaStream_t)stream;
  if (p->n_tokens == 0 || p->n_req == 0)
    return cudaMemsetAsync(ws, 0, sizeof(uint32_t), st) == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
  const bool is_wide = wide(p, sms);
  Params P = params_of(c, p, L, is_wide);
  set_clusters(P, p, L.max_tiles, sms);
  const auto plan_smem = [](int n_req) { return (size_t)(n_req + 1) * 2 * sizeof(long long); };
  const size_t smem = plan_smem(p->n_req), most_smem = plan_smem(DSA_KV8_MAX_REQ);
  const int rc1 = P.own_plan ? launch(plan_kernel<FEW_THREADS>, 1, FEW_THREADS, smem, most_smem, st, P, false)
                             : launch(plan_kernel<PLAN_THREADS>, 1, PLAN_THREADS, smem, most_smem, st, P, false);
  if (rc1 != DSA_OK) return rc1;
  return p->d == 128 ? launch_all<128>(p, P, is_wide, st) : launch_all<64>(p, P, is_wide, st);
}

}  // extern "C"
