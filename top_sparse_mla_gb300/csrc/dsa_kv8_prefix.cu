// Attention over the paged 8-bit cache for requests that share a prefix (include/dsa_kv8_prefix.h).
//
// The queries of a group see the pages that its requests share all alike, so that they are rows of one
// problem there: the shared pages are read once for them and, where they are more than rows_kernel takes,
// go to the tensor cores in tiles.  What a request sees behind the shared pages is a problem of its own.
// The plan kernel finds both kinds (find_parts); the kernels of dsa_kv8_attn_fwd take them
// (dsa_kv8_rows.cuh, dsa_kv8_tiles.cuh) and leave each row's O, m and l of either part in the
// workspace; a last kernel joins the two.

#include "dsa_kv8_prefix.h"

#include "dsa_kv8_rows.cuh"

namespace dsa_kv8 {
constexpr int LAUNCH_REGS = 128;   // of a thread of the tiles' kernel
}

#include "dsa_kv8_tiles.cuh"

namespace dsa_kv8 {

// ------------------------------------------------------------------------------ join
// CTAs (x, r) have the query rows of request r; a thread takes 8 dims of a row at a time.
constexpr int JOIN_THREADS = 256, JOIN_TRIPS = 4;
template <int D>
__global__ void __launch_bounds__(JOIN_THREADS) join_kernel(const __grid_constant__ Params P) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Request a = request<true>(P, P.n_groups + blockIdx.y);
  const bool both = a.lo > 0;
  const long long items = (long long)a.q_len * P.h_q * (D / 8);
  for (long long u = (long long)blockIdx.x * JOIN_THREADS + threadIdx.x; u < items; u += (long long)gridDim.x * JOIN_THREADS) {
    const int k = (int)(u % (D / 8)) * 8;
    const long long row = u / (D / 8);
    const int i = (int)(row / P.h_q), head = (int)(row - (long long)i * P.h_q), token = a.q0 + i;
    float m = 0.f, l = 0.f, o[8];
    float2 ml[2];
    float4 v[2][2];
#pragma unroll
    for (int side = SHARED; side <= OWN; ++side) {
      ml[side] = make_float2(M_INIT, 0.f);
      v[side][0] = v[side][1] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (side == OWN || both) {
        const long long at = part_row(P, side, token, head);
        ml[side] = P.part_ml[at];
        const float4* from = reinterpret_cast<const float4*>(P.part_o + at * D + k);
        v[side][0] = from[0];
        v[side][1] = from[1];
      }
    }
    m = fmaxf(ml[0].x, ml[1].x);
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = 0.f;
#pragma unroll
    for (int side = SHARED; side <= OWN; ++side) {
      const float f = ex2(ml[side].x - m);
      l += scaled(ml[side].y, ml[side].x - m);
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        o[4 * q] = fmaf(v[side][q].x, f, o[4 * q]);
        o[4 * q + 1] = fmaf(v[side][q].y, f, o[4 * q + 1]);
        o[4 * q + 2] = fmaf(v[side][q].z, f, o[4 * q + 2]);
        o[4 * q + 3] = fmaf(v[side][q].w, f, o[4 * q + 3]);
      }
    }
    const float inv = l > 0.f ? 1.0f / l : (l == 0.f ? 0.f : l);   // a NaN sum stays one
    uint4 w;
    w.x = pack(o[0] * inv, o[1] * inv, P.fp16);
    w.y = pack(o[2] * inv, o[3] * inv, P.fp16);
    w.z = pack(o[4] * inv, o[5] * inv, P.fp16);
    w.w = pack(o[6] * inv, o[7] * inv, P.fp16);
    *reinterpret_cast<uint4*>(P.out + token * P.out_ld + head * P.out_hd + k) = w;
    if (k == 0 && P.lse) P.lse[(long long)token * P.h_q + head] = l == 0.f ? -INFINITY : 0.6931471805599453f * (m + log2f(l));
  }
}

// ------------------------------------------------------------------------------ host
static int check_prefix(const dsa_kv8_params* p, int n_groups) {
  const int rc = check(p);
  if (rc != DSA_OK) return rc;
  if (n_groups < 0) return DSA_ERR_INVALID_ARG;
  return p->window > 0 || n_groups > DSA_KV8_MAX_REQ - p->n_req ? DSA_ERR_UNSUPPORTED_SHAPE : DSA_OK;
}

struct PrefixLayout {
  Layout base;
  size_t parts, part_o, part_ml, bytes;
};

static PrefixLayout prefix_layout(const dsa_kv8_params* p, int n_groups, int sms) {
  PrefixLayout L;
  const size_t group = p->h_q / p->h_kv, rows = 8 * (size_t)row_tiles(p), queries = (size_t)p->n_tokens * p->h_q;
  Layout& b = L.base;
  b.n_shares = ctas_per_sm(p->d, row_tiles(p)) * sms;
  // ascending cu_q and cu_groups cannot give more
  b.max_tiles = (int)((p->n_tokens * group + (TILE_ROWS - 1) * (size_t)n_groups) / TILE_ROWS);
  if (has_tiles(p)) b.max_tiles += (int)((p->n_tokens * group + (TILE_ROWS - 1) * (size_t)p->n_req) / TILE_ROWS);
  size_t at = 256;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += up(bytes);
    return here;
  };
  b.shares = take(b.n_shares * sizeof(Share));
  b.arrived = take(b.n_shares * 3 * sizeof(int));
  b.tiles = take((size_t)b.max_tiles * sizeof(Tile));
  b.partial = take((size_t)b.n_shares * 4 * (rows * p->d + 2 * rows) * sizeof(float));
  L.parts = take((size_t)(p->n_req + n_groups) * sizeof(Part));
  L.part_o = take(2 * queries * p->d * sizeof(float));
  L.part_ml = take(2 * queries * sizeof(float2));
  L.bytes = b.bytes = at;
  return L;
}

template <int D>
static int launch_prefix(const dsa_kv8_params* p, const Params& P, cudaStream_t st) {
  const int nt = row_tiles(p);
  int rc = nt == 1 ? launch_rows<D, 1, true>(P, false, st) : nt == 2 ? launch_rows<D, 2, true>(P, false, st) : launch_rows<D, 4, true>(P, false, st);
  if (rc == DSA_OK && P.has_tiles) rc = launch_tiles_of<true>(D, P, st);
  if (rc != DSA_OK) return rc;
  cudaLaunchConfig_t cfg = {};
  const long long items = (long long)p->max_q_len * p->h_q * (D / 8), trip = JOIN_THREADS * JOIN_TRIPS;
  const long long most = 2LL * P.n_shares, x = (items + trip - 1) / trip;
  cfg.gridDim = dim3((unsigned)(x < 1 ? 1 : x > most ? most : x), (unsigned)p->n_req);
  cfg.blockDim = dim3(JOIN_THREADS);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, join_kernel<D>, P) == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}

}  // namespace dsa_kv8

extern "C" {

size_t dsa_kv8_prefix_workspace_size(const dsa_kv8_params* p, int32_t n_groups, int num_sms) {
  if (dsa_kv8::check_prefix(p, n_groups) != DSA_OK) return 0;
  if (num_sms <= 0 && dsa_kv8::current_sms(&num_sms) != DSA_OK) return 0;
  return dsa_kv8::prefix_layout(p, n_groups, num_sms).bytes;
}

int dsa_kv8_prefix_attn_fwd(const void* q, int64_t q_ld, int64_t q_hd, const void* k_pool, const void* v_pool,
                            const float* k_scale, const float* v_scale, const int32_t* block_table, int64_t table_ld,
                            const int32_t* cu_q, const int32_t* kv_lens, const int32_t* cu_groups, const int32_t* prefix_lens,
                            int32_t n_groups, void* out, int64_t out_ld, int64_t out_hd, float* lse,
                            const dsa_kv8_params* p, void* workspace, size_t workspace_bytes, void* stream) {
  using namespace dsa_kv8;
  const int rc = check_prefix(p, n_groups);
  if (rc != DSA_OK) return rc;
  const Call c{q, q_ld, q_hd, k_pool, v_pool, k_scale, v_scale, block_table, table_ld, cu_q, kv_lens, out, out_ld, out_hd, lse, workspace};
  if (bad_call(c, p)) return DSA_ERR_INVALID_ARG;
  if (n_groups > 0 && (!cu_groups || !prefix_lens || !aligned(cu_groups, 4) || !aligned(prefix_lens, 4))) return DSA_ERR_INVALID_ARG;
  int sms = 0;
  const int rc0 = gb300_sms(&sms);
  if (rc0 != DSA_OK) return rc0;
  const PrefixLayout L = prefix_layout(p, n_groups, sms);
  if (workspace_bytes < L.bytes) return DSA_ERR_WORKSPACE_TOO_SMALL;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  cudaStream_t st = (cudaStream_t)stream;
  if (p->n_tokens == 0 || p->n_req == 0)
    return cudaMemsetAsync(ws, 0, sizeof(uint32_t), st) == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
  Params P = params_of(c, p, L.base, sms, false);
  P.n_req = p->n_req + n_groups;
  P.parts = reinterpret_cast<Part*>(ws + L.parts);
  P.cu_groups = cu_groups;
  P.prefix_lens = prefix_lens;
  P.part_o = reinterpret_cast<float*>(ws + L.part_o);
  P.part_ml = reinterpret_cast<float2*>(ws + L.part_ml);
  P.n_groups = n_groups;
  P.own_plan = 0;
  P.has_tiles = L.base.max_tiles > 0;
  set_clusters(P, p, L.base.max_tiles, sms);
  const size_t smem = (size_t)(P.n_req + 1) * 2 * sizeof(long long) + 2 * (size_t)n_groups * sizeof(int);
  const size_t most = (size_t)(DSA_KV8_MAX_REQ + 1) * 2 * sizeof(long long) + 2 * (size_t)DSA_KV8_MAX_REQ * sizeof(int);
  static_assert((DSA_KV8_MAX_REQ + 1) * 16 + DSA_KV8_MAX_REQ * 8 + 8 * 1024 <= 227 * 1024, "shared memory of the plan");
  const int rc1 = P.n_req <= 2 * FEW_THREADS ? launch(plan_kernel<FEW_THREADS, true>, 1, FEW_THREADS, smem, most, st, P, false)
                                             : launch(plan_kernel<PLAN_THREADS, true>, 1, PLAN_THREADS, smem, most, st, P, false);
  if (rc1 != DSA_OK) return rc1;
  return p->d == 128 ? launch_prefix<128>(p, P, st) : launch_prefix<64>(p, P, st);
}

}  // extern "C"
