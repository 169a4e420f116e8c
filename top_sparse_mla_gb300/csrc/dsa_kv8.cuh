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
  int req, row0;
  int q0, rows;      // the request's first query token and its rows
  int pos0;          // position of its first query
  int lo, hi;        // cached tokens that the tile's rows see, lo rounded down to a step
  int pad;
};

struct Header {
  uint32_t status;
  int n_tiles;
  long long share;   // steps of every CTA
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
  uint32_t test_block;   // block of CTA 0 at which the copies stop (DSA_KV8_FLAG_TEST_WAIT_TIMEOUT)
  float scale_log2;   // softmax_scale * log2 e
};

struct Request {
  int q0, q_len, kv;
  __device__ __forceinline__ int rows(const Params& P) const { return q_len * P.group; }
};

__device__ __forceinline__ Request request(const Params& P, int from, int to, int kv_len) {
  Request a;
  a.q0 = min(max(from, 0), P.n_tokens);
  a.q_len = min(max(to, a.q0), P.n_tokens) - a.q0;
  a.kv = min(max(kv_len, 0), P.cap);
  return a;
}
__device__ __forceinline__ Request request(const Params& P, int r) {
  return request(P, P.cu_q[r], P.cu_q[r + 1], P.kv_lens[r]);
}

// The cached tokens [lo, hi) that the query positions [p0, p1] may see, lo rounded down to
// a step.  Never empty: a row that sees nothing is still computed, and its result is 0.
struct Span {
  int lo, steps;
};
__device__ __forceinline__ Span span(const Params& P, const Request& a, int i0, int i1) {
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
