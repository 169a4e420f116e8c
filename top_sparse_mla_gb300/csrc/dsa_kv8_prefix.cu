// Attention over the paged 8-bit cache for requests that share a prefix (include/dsa_kv8_prefix.h).
//
// The queries of a group see the pages that its requests share all alike, so that they are rows of one
// problem there: the shared pages are read once for them and, where they are more than rows_kernel takes,
// go to the tensor cores in tiles.  What a request sees behind the shared pages is a problem of its own.
// The plan kernel finds both kinds (find_parts); the kernels of dsa_kv8_attn_fwd take them
// (dsa_kv8_rows.cuh, dsa_kv8_tiles.cuh) and leave each row's O, m and l of either part in the
// workspace; a last kernel joins the two.

#include <atomic>

#include "device.cuh"
#include "dsa_kv8_prefix.h"

#include "dsa_kv8_rows.cuh"

namespace dsa_kv8 {
constexpr int LAUNCH_REGS = 128;   // of a thread of the tiles' kernel
}

#include "dsa_kv8_tiles.cuh"

namespace dsa_kv8 {

// ------------------------------------------------------------------------------ join
// A thread takes 8 dims of a row at a time.  The pieces of a part are joined in their order, and then the
// parts.  By request: CTAs (x, r) have the rows of request r, as many of them as max_q_len asks for; else the
// CTAs have those of the batch and each row looks for its request.  launch_prefix() chooses.
constexpr int JOIN_THREADS = 256;

constexpr int AT_ONCE = 4;   // pieces on their way together

struct Sum {   // of a row: O and l in units of 2^m
  float m, l, o[8];
  template <int N>
  __device__ __forceinline__ void add(const float (&m1)[N], const float (&l1)[N], const float4 (&v)[N][2]) {
    float top = m;
#pragma unroll
    for (int j = 0; j < N; ++j) top = fmaxf(top, m1[j]);
    l = scaled(l, m - top);
    const float f0 = ex2(m - top);
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] *= f0;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      if (m1[j] == NOTHING && l1[j] == 0.f) continue;   // O is not written
      const float f = ex2(m1[j] - top);
      l += scaled(l1[j], m1[j] - top);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        o[4 * h] = fmaf(v[j][h].x, f, o[4 * h]);
        o[4 * h + 1] = fmaf(v[j][h].y, f, o[4 * h + 1]);
        o[4 * h + 2] = fmaf(v[j][h].z, f, o[4 * h + 2]);
        o[4 * h + 3] = fmaf(v[j][h].w, f, o[4 * h + 3]);
      }
    }
    m = top;
  }
};

template <int D>
__device__ __forceinline__ void add_part(const Params& P, const Part& a, int n_tiles, int token, int head, int k, Sum& sum) {
  if (a.q_len * P.group > P.small_rows && P.tile_shares) {
    const int row = (token - a.q0) * P.group + head % P.group, tile = a.tile0 + row / TILE_ROWS, r = row % TILE_ROWS;
    if ((unsigned)tile >= (unsigned)n_tiles) return;   // lists that do not ascend may give more tiles than there is room for
    const int2 by = P.unit_ctas[tile * P.h_kv + head / P.group];
    if (by.x != by.y) {
      for (int b0 = by.x; b0 <= by.y; b0 += AT_ONCE) {
        float m[AT_ONCE], l[AT_ONCE];
        float4 v[AT_ONCE][2];
#pragma unroll
        for (int j = 0; j < AT_ONCE; ++j) {
          m[j] = NOTHING;
          l[j] = 0.f;
          v[j][0] = v[j][1] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (b0 + j <= by.y) {
            const float* piece = P.pieces + (2LL * (b0 + j) + (b0 + j == by.x ? 1 : 0)) * piece_size(D);
            m[j] = piece[TILE_ROWS * D + r];
            l[j] = piece[TILE_ROWS * (D + 1) + r];
            const float4* o = reinterpret_cast<const float4*>(piece + (k / 4 * TILE_ROWS + r) * 4);
            v[j][0] = o[0];
            v[j][1] = o[TILE_ROWS];
          }
        }
        sum.add(m, l, v);
      }
      return;
    }
  }
  const long long at = part_row(P, a.side, token, head);
  const float2 ml = P.part_ml[at];
  const float4* o = reinterpret_cast<const float4*>(P.part_o + at * D + k);
  const float m[1] = {ml.x}, l[1] = {ml.y};
  const float4 v[1][2] = {{o[0], o[1]}};
  sum.add(m, l, v);
}

template <int D, bool BY_REQUEST>
__global__ void __launch_bounds__(JOIN_THREADS) join_kernel(const __grid_constant__ Params P) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int n_tiles = P.header->n_tiles, n = P.n_req - P.n_groups;
  // a graph's next launch has the same number
  if (blockIdx.x + blockIdx.y + threadIdx.x == 0) P.header->planned = 0;
  int r = BY_REQUEST ? blockIdx.y : 0;
  Part own = P.parts[P.n_groups + r], shared = P.parts[own.lo > 0 ? own.group : P.n_groups + r];
  const long long items = (long long)(BY_REQUEST ? own.q_len : P.n_tokens) * P.h_q * (D / 8);
  for (long long u = (long long)blockIdx.x * JOIN_THREADS + threadIdx.x; u < items; u += (long long)gridDim.x * JOIN_THREADS) {
    // the heads of a KV head side by side, as their rows are in a piece
    const long long v = u / P.group, row = v / (D / 8);
    const int k = (int)(v % (D / 8)) * 8, i = (int)(row / P.h_kv), token = BY_REQUEST ? own.q0 + i : i;
    const int head = (int)(row - (long long)i * P.h_kv) * P.group + (int)(u - v * P.group);
    if (!BY_REQUEST) {
      int hi = n;   // the last request that begins at or before the token
      r = 0;
      while (hi - r > 1) {
        const int mid = (r + hi) >> 1;
        if (min(max(__ldg(P.cu_q + mid), 0), P.n_tokens) <= token) r = mid; else hi = mid;
      }
      own = P.parts[P.n_groups + r];
      if (token < own.q0 || token >= own.q0 + own.q_len) continue;   // of no request, or of one that is skipped
      shared = P.parts[own.lo > 0 ? own.group : P.n_groups + r];
    }
    Sum s;
    s.m = M_INIT;
    s.l = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) s.o[e] = 0.f;
    if (own.lo > 0) add_part<D>(P, shared, n_tiles, token, head, k, s);
    add_part<D>(P, own, n_tiles, token, head, k, s);
    const float inv = s.l > 0.f ? 1.0f / s.l : (s.l == 0.f ? 0.f : s.l);   // a NaN sum stays one
    uint4 w;
    w.x = pack(s.o[0] * inv, s.o[1] * inv, P.fp16);
    w.y = pack(s.o[2] * inv, s.o[3] * inv, P.fp16);
    w.z = pack(s.o[4] * inv, s.o[5] * inv, P.fp16);
    w.w = pack(s.o[6] * inv, s.o[7] * inv, P.fp16);
    *reinterpret_cast<uint4*>(P.out + token * P.out_ld + head * P.out_hd + k) = w;
    if (k == 0 && P.lse) P.lse[(long long)token * P.h_q + head] = s.l == 0.f ? -INFINITY : 0.6931471805599453f * (s.m + log2f(s.l));
  }
}

// ------------------------------------------------------------------------------ host
static int check_prefix(const dsa_kv8_params* p, int n_groups) {
  const int rc = check(p);
  if (rc != DSA_OK) return rc;
  if (n_groups < 0) return DSA_ERR_INVALID_ARG;
  return p->window > 0 || n_groups > DSA_KV8_MAX_GROUPS || n_groups > DSA_KV8_MAX_REQ - p->n_req ? DSA_ERR_UNSUPPORTED_SHAPE : DSA_OK;
}

struct PrefixLayout {
  Layout base;
  bool tile_shares;
  size_t parts, row_parts, part_o, part_ml, tile_steps, tile_cuts, cut_units, unit_ctas, pieces, bytes;
};

// Tiles and heads of an SM below which the tiles' blocks are shared out to all SMs alike, whatever their
// lengths; with more of them, whole ones keep the SMs as busy.
constexpr int SHARE_UNITS = 2;
constexpr int MOST_SHARED_TILES = 1024;   // for the plan's shared memory

// All query rows of the batch by KV head, where rows_kernel can take them: no tiles then
static int batch_rows(const dsa_kv8_params* p) {
  const long long rows = (long long)p->n_tokens * (p->h_q / p->h_kv);
  return rows <= MAX_ROWS ? (int)rows : 0;
}
static int prefix_row_tiles(const dsa_kv8_params* p) {
  const int rows = batch_rows(p);
  return rows == 0 ? row_tiles(p) : rows <= 8 ? 1 : rows <= 16 ? 2 : 4;
}

static PrefixLayout prefix_layout(const dsa_kv8_params* p, int n_groups, int sms) {
  PrefixLayout L;
  const size_t group = p->h_q / p->h_kv, rows = 8 * (size_t)prefix_row_tiles(p), queries = (size_t)p->n_tokens * p->h_q;
  Layout& b = L.base;
  b.n_shares = ctas_per_sm(p->d, prefix_row_tiles(p)) * sms;
  // ascending cu_q and cu_groups cannot give more
  b.max_tiles = (int)((p->n_tokens * group + (TILE_ROWS - 1) * (size_t)n_groups) / TILE_ROWS);
  if (batch_rows(p) > 0 || n_groups + p->n_req == 0) b.max_tiles = 0;
  else if (has_tiles(p)) b.max_tiles += (int)((p->n_tokens * group + (TILE_ROWS - 1) * (size_t)p->n_req) / TILE_ROWS);
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
  L.row_parts = take((size_t)(p->n_req + n_groups) * sizeof(int));
  L.part_o = take(2 * queries * p->d * sizeof(float));
  L.part_ml = take(2 * queries * sizeof(float2));
  const long long blocks = ((long long)p->table_cols * p->page_size + TILE_BLOCK - 1) / TILE_BLOCK + 1;   // of a tile at most
  L.tile_shares = b.max_tiles > 0 && b.max_tiles < MOST_SHARED_TILES && (long long)b.max_tiles * p->h_kv < SHARE_UNITS * (long long)sms &&
                  sms < 256 && blocks <= (1 << 24) && blocks * b.max_tiles * p->h_kv < (1 << 30);   // the plan's 32 bits
  L.tile_steps = take(L.tile_shares ? (b.max_tiles + 1) * sizeof(long long) : 0);
  L.tile_cuts = take(L.tile_shares ? (sms + 1) * sizeof(long long) : 0);
  L.cut_units = take(L.tile_shares ? sms * sizeof(int) : 0);
  L.unit_ctas = take(L.tile_shares ? (size_t)b.max_tiles * p->h_kv * sizeof(int2) : 0);
  L.pieces = take(L.tile_shares ? 2 * (size_t)sms * piece_size(p->d) * sizeof(float) : 0);
  L.bytes = b.bytes = at;
  return L;
}

template <int D>
static int launch_prefix(const dsa_kv8_params* p, const Params& P, cudaStream_t st) {
  const int nt = prefix_row_tiles(p);
  int rc = nt == 1 ? launch_rows<D, 1, true>(P, false, st) : nt == 2 ? launch_rows<D, 2, true>(P, false, st) : launch_rows<D, 4, true>(P, false, st);
  if (rc == DSA_OK && P.has_tiles) rc = launch_tiles_of<true>(D, P, st);
  if (rc != DSA_OK) return rc;
  cudaLaunchConfig_t cfg = {};
  // By request where that is at most twice the CTAs that the batch's rows need: the search takes 1 to 2.5 us (4 requests
  // behind 2k 20.6 and 21.6, 64 behind 16k 76.0 and 78.7, 240 verified 51.4 and 52.9).  But 4096 requests of one query
  // behind 256 tokens, 16/2 heads, take 5684 by request where max_q_len is n_tokens, and 182 without; 64 decoded
  // requests beside a chunk of 2048 queries 266 and 197.
  const long long most = 2LL * P.n_shares, per_query = (long long)p->h_q * (D / 8);
  auto needed = [&](long long queries) { return (queries * per_query + JOIN_THREADS - 1) / JOIN_THREADS; };
  auto grid = [&](long long queries) {
    const long long x = needed(queries);
    return x < 1 ? 1 : x > most ? most : x;
  };
  const bool by_request = grid(p->max_q_len) * p->n_req <= 2 * needed(p->n_tokens);
  cfg.gridDim = by_request ? dim3((unsigned)grid(p->max_q_len), (unsigned)p->n_req) : dim3((unsigned)grid(p->n_tokens));
  cfg.blockDim = dim3(JOIN_THREADS);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t rc1 = by_request ? cudaLaunchKernelEx(&cfg, join_kernel<D, true>, P) : cudaLaunchKernelEx(&cfg, join_kernel<D, false>, P);
  return rc1 == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}

}  // namespace dsa_kv8

extern "C" {

size_t dsa_kv8_prefix_workspace_size(const dsa_kv8_params* p, int32_t n_groups, int num_sms) {
  if (dsa_kv8::check_prefix(p, n_groups) != DSA_OK) return 0;
  if (num_sms <= 0 && dsa::current_sms(&num_sms) != DSA_OK) return 0;
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
  const int rc0 = dsa::gb300_sms(&sms);
  if (rc0 != DSA_OK) return rc0;
  const PrefixLayout L = prefix_layout(p, n_groups, sms);
  if (workspace_bytes < L.bytes) return DSA_ERR_WORKSPACE_TOO_SMALL;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  cudaStream_t st = (cudaStream_t)stream;
  if (p->n_tokens == 0 || p->n_req == 0)
    return cudaMemsetAsync(ws, 0, sizeof(uint32_t), st) == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
  Params P = params_of(c, p, L.base, false);
  P.n_req = p->n_req + n_groups;
  P.parts = reinterpret_cast<Part*>(ws + L.parts);
  P.row_parts = reinterpret_cast<int*>(ws + L.row_parts);
  P.cu_groups = cu_groups;
  P.prefix_lens = prefix_lens;
  P.part_o = reinterpret_cast<float*>(ws + L.part_o);
  P.part_ml = reinterpret_cast<float2*>(ws + L.part_ml);
  P.n_groups = n_groups;
  static std::atomic<uint32_t> calls{0};
  // the upper half: a workspace may have anything in it at first
  P.call = 0x706C616Eull << 32 | calls.fetch_add(1, std::memory_order_relaxed);
  P.most_shared = (int)(MOST_TOKENS - p->n_tokens);
  P.own_plan = 0;
  P.small_rows = 8 * prefix_row_tiles(p);
  P.has_tiles = L.base.max_tiles > 0;
  P.cluster = 0;
  P.n_ctas = sms;
  P.tile_shares = L.tile_shares;
  P.tile_steps = reinterpret_cast<long long*>(ws + L.tile_steps);
  P.tile_cuts = reinterpret_cast<long long*>(ws + L.tile_cuts);
  P.cut_units = reinterpret_cast<int*>(ws + L.cut_units);
  P.unit_ctas = reinterpret_cast<int2*>(ws + L.unit_ctas);
  P.pieces = reinterpret_cast<float*>(ws + L.pieces);
  // the plan's lists of parts, and the groups' (find_parts) or the shared out tiles'
  const auto plan_smem = [](size_t parts, size_t groups, size_t tiles) {
    const size_t g = (3 * groups + 1) * sizeof(int), t = 3 * tiles * sizeof(int);
    return (parts + 1) * 2 * sizeof(long long) + (g > t ? g : t);
  };
  const size_t smem = plan_smem(P.n_req, n_groups, L.tile_shares ? L.base.max_tiles + 1 : 0);
  const size_t most = plan_smem(DSA_KV8_MAX_REQ, DSA_KV8_MAX_GROUPS, MOST_SHARED_TILES + 1);
  static_assert((DSA_KV8_MAX_REQ + 1) * 16 + (3 * DSA_KV8_MAX_GROUPS + 1) * 4 + 8 * 1024 <= 227 * 1024, "shared memory of the plan");
  const int rc1 = P.n_req <= 2 * FEW_THREADS ? launch(plan_kernel<FEW_THREADS, true>, 1, FEW_THREADS, smem, most, st, P, false)
                                             : launch(plan_kernel<PLAN_THREADS, true>, 1, PLAN_THREADS, smem, most, st, P, false);
  if (rc1 != DSA_OK) return rc1;
  return p->d == 128 ? launch_prefix<128>(p, P, st) : launch_prefix<64>(p, P, st);
}

}  // extern "C"
