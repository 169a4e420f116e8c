// What the kernels of the attention over the paged 8-bit cache share (dsa_kv8_attn.cu,
// dsa_kv8_tiles.cu): the parameters, a request's rows and the positions that they see.
#pragma once

#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "dsa_kv8.h"
#include "ptx_sm103.cuh"

namespace dsa_kv8 {

constexpr int STEP = 16;          // cached tokens of one step of a warp; every page size is a multiple
constexpr int TILE_ROWS = 256;    // query rows of a tile
constexpr int TILE_BLOCK = 128;   // cached tokens of a tile's block
constexpr int MAX_CLUSTER = 16;
// The softmax's sum is that of w / v_scale, but where pages' value scales are so far apart that a w may
// be too small for fp32: there it is that of 2^(score - maximum).  rows_kernel goes by each page's
// scale, the tiles by the largest and the least of a unit, whose scores they form once more.  us, with
// and without: 1024 windowed requests 44.4 and 43.9, 48 verified 89.5 and 88.9, one of 32k 20.1 and
// 19.8; a 2123-token prefill 96.0 and 95.1, 6 chunks 690 and 686.
constexpr float SMALL_SCALE = 2.3283064365386963e-10f;   // 2^-32
constexpr float FAR_APART = 1.2379400392853803e27f;      // 2^90: w stays a normal number for every p above 2^-36
constexpr float LAG = 8.0f;       // how far, in powers of two, a running maximum may lag

struct Share {   // where a CTA's share of the steps begins
  int req, head;
  long long step;
};

struct Tile {   // rows [row0, row0 + TILE_ROWS) of a request (query * group + head of the group)
  int req, row0;     // req: row of the block table
  int q0, rows;      // the request's first query token and its rows
  int pos0;          // position of its first query
  int lo, hi;        // cached tokens that the tile's rows see, lo rounded down to a step
  int side;          // PREFIX: which part of its rows' tokens these are, SHARED or OWN
};

struct Header {
  uint32_t status;
  int n_tiles;
  long long share;   // steps of every CTA
  int row_units;     // PREFIX: units that rows_kernel's CTAs take whole, one after the other; 0 where they have shares
  int next_unit;     // how many were taken beside each CTA's first
  unsigned long long planned;   // PREFIX: the call's number once its plan is there, and 0 in the end
};

enum { SHARED = 0, OWN = 1 };
// What the rows of a group, or of a request, see of the cache in one part: tokens [lo, hi) by block table row
// `req`, and of those the ones up to their own positions, pos0 for the first query.
struct Part {
  int q0, q_len, pos0, lo;
  int hi, req, side, group;   // group: of a request's own part, or -1
  int tile0, pad[3];          // the first of its tiles, where it has some
};

struct Params {
  const uint16_t* q;
  const uint8_t *k_pool, *v_pool;
  const float *k_scale, *v_scale;
  const int32_t *table, *cu_q, *kv_lens;
  uint16_t* out;
  float* lse;
  long long q_ld, q_hd, out_ld, out_hd, table_ld;
  Header* header;
  Share* shares;
  int* arrived;
  Tile* tiles;
  float* partial;
  int n_tokens, n_req, h_q, h_kv, group, n_pages, page_shift, cap, max_q_len, window, fp16;
  int small_rows;   // requests with at most this many rows go to rows_kernel
  int unit_steps, min_share;   // what a unit costs a CTA beside its steps, and a CTA's least share, in steps
  int own_plan;     // requests of a thread where rows_kernel's CTAs find their shares for themselves, else 0
  int n_shares, max_tiles, n_ctas;   // n_ctas: of the tiles' kernel
  int has_tiles;    // whether requests may have more rows than rows_kernel takes
  int cluster;      // CTAs that share a tile and KV head; 0: a CTA has several of them
  // Requests that share a prefix (dsa_kv8_prefix.cu): n_req counts the groups and the requests, whose
  // parts are in `parts`; the queries' O, m and l of either part go to part_o and part_ml
  Part* parts;
  const int32_t *cu_groups, *prefix_lens;
  float* part_o;
  float2* part_ml;
  // Tiles whose blocks are shared out (PREFIX and SPLIT): all blocks, of all heads of all tiles, lie in a row.  The ones in
  // front of each tile, by head; where each CTA's begin, with the unit that is there; and the first and last CTA of each unit.
  // m, l and O of a CTA's two pieces: of a unit that it continued (0), and of one that it began (1)
  long long *tile_steps, *tile_cuts;
  int* cut_units;
  int2* unit_ctas;
  float* pieces;
  int* row_parts;   // parts of rows_kernel whose units are taken whole
  int n_groups, tile_shares;
  unsigned long long call;   // another number for every call, never 0
  int most_shared;   // tokens of a group: its rows' positions go on from the last one, and stay as far below 2^31 as others
  uint32_t test_block;   // block of CTA 0 at which the copies stop (DSA_KV8_FLAG_TEST_WAIT_TIMEOUT)
  float scale_log2;   // softmax_scale * log2 e
};

struct Request {
  int q0, q_len, kv;
  int lo, hi, req, side;   // PREFIX
  __device__ __forceinline__ int rows(const Params& P) const { return q_len * P.group; }
};

__device__ __forceinline__ Request request(const Params& P, int from, int to, int kv_len) {
  Request a;
  a.q0 = min(max(from, 0), P.n_tokens);
  a.q_len = min(max(to, a.q0), P.n_tokens) - a.q0;
  a.kv = min(max(kv_len, 0), P.cap);
  return a;
}
template <bool PREFIX = false>
__device__ __forceinline__ Request request(const Params& P, int r) {
  if (!PREFIX) return request(P, P.cu_q[r], P.cu_q[r + 1], P.kv_lens[r]);
  // plain loads: the plan writes them while the kernels that read them are there already
  const int4* at = reinterpret_cast<const int4*>(P.parts + r);
  const int4 x = at[0], y = at[1];
  Request a;
  a.q0 = x.x; a.q_len = x.y; a.kv = x.z + x.y;
  a.lo = x.w; a.hi = y.x; a.req = y.y; a.side = y.z;
  return a;
}
// floats of a piece: O in the order [d / 4][row][4], m, l
__device__ __host__ __forceinline__ size_t piece_size(int d) { return (size_t)TILE_ROWS * (d + 2); }
// a query row's place in part_o and part_ml
__device__ __forceinline__ long long part_row(const Params& P, int side, int token, int head) {
  return ((long long)side * P.n_tokens + token) * P.h_q + head;
}

// The cached tokens [lo, hi) that the query positions [p0, p1] may see, lo rounded down to
// a step.  Never empty: a row that sees nothing is still computed, and its result is 0.
struct Span {
  int lo, steps;
};
template <bool PREFIX = false>
__device__ __forceinline__ Span span(const Params& P, const Request& a, int i0, int i1) {
  if (PREFIX) {   // no window, and a part begins at a step
    const int end = min(a.kv - a.q_len + i1 + 1, a.hi);
    return Span{a.lo, max((end - a.lo + STEP - 1) / STEP, 1)};
  }
  const int p0 = a.kv - a.q_len + i0, p1 = a.kv - a.q_len + i1;
  Span s;
  s.lo = P.window > 0 ? max(p0 - P.window + 1, 0) & ~(STEP - 1) : 0;
  s.steps = max((p1 + 1 - s.lo + STEP - 1) / STEP, 1);
  if (p1 + 1 <= s.lo) s.steps = 1;
  return s;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// v 2^d, also where 2^d is below fp32's range and v 2^d is not: a softmax's sum in units of
// 2^maximum may be 2^64 and more (the maximum has a page's value scale in it, the sum has not).
__device__ __forceinline__ float scaled(float v, float d) {
  const float h = ex2(0.5f * d);
  return v * h * h;
}

__device__ __forceinline__ uint32_t word(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

__device__ __forceinline__ float2 unpack(uint32_t w, int fp16) {
  if (fp16) return __half22float2(*reinterpret_cast<const __half2*>(&w));
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
__device__ __forceinline__ uint32_t pack(float a, float b, int fp16) {
  if (fp16) return dsa::pack_f16x2(a, b);
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}

// The power of two 2^-e that brings a row's largest magnitude to [2^7, 2^8), where the
// row's values are exact in fp16 down to 2^-25 of the largest with bf16's significands and
// 2^-22 with fp16's; `back` is 2^e.  Both stay normal numbers.
__device__ __forceinline__ float row_scaling(float largest, float& back) {
  const int e = largest > 0.f ? min(max((int)(__float_as_uint(largest) >> 23) - 127 - 7, -100), 120) : 0;
  back = __uint_as_float((uint32_t)(127 + e) << 23);
  return __uint_as_float((uint32_t)(127 - e) << 23);
}

// A page's value scale within [2^-64, 2^64]
__device__ __forceinline__ float bounded_scale(float s) {
  return fminf(fmaxf(s, 5.421010862427522e-20f), 1.8446744073709552e19f);
}

// dsa_kv8_tiles.cu: the tiles of the requests with more rows than rows_kernel takes
// How many CTAs should share each of at most `units` pairs of a tile and a KV head, with at
// most `blocks` blocks of 128 cached tokens: 0 for one CTA alone.
int cluster_size(int d, long long units, int blocks);
int launch_tiles(int d, const Params& P, cudaStream_t st);

}  // namespace dsa_kv8
