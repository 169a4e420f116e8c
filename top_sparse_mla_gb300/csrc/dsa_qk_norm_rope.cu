// RMS norm and rotation of the heads of queries and keys (include/dsa_qk_norm_rope.h).
//
// What bounds it: memory, each value read and written once.  A row (token, head) belongs to G lanes of 16
// values each, two 16-byte parts: of a rotary half and of the other half what turns with it, so that a lane
// has both values of its pairs; or, interleaved and behind the rotary values, neighbours.  A lane group goes
// through heads of one token and forms the cosines and sines of its lanes' pairs once, in registers, while
// its first rows are on their way.  (Kept in shared memory for the CTA's tokens and read with every row, and
// with a lane's values side by side and their partners exchanged by shuffles, both through one pipe, 16381
// tokens of 64 + 8 heads of 128 took 198 us against 104.6 now, 5.8 TB/s, 0.85 of a copy.)
//
// The angle of pair i is position * turns[i] in 64-bit fixed point, a fraction of a turn that
// wraps by itself: an fp32 angle would be off by 2^-24 of itself, half a turn at position 2^24.

#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "device.cuh"
#include "dsa_qk_norm_rope.h"
#include "ptx_sm103.cuh"

namespace dsa_qk {

constexpr int THREADS = 256;
constexpr int MAX_PAIRS = 128;     // rotary pairs of a head
constexpr int AT_ONCE = 4;         // rows of a lane group in flight
constexpr int MOST_ROWS = 32;      // heads that a lane group goes through with one token's angles, at most
constexpr int SPREAD = 4, ANGLE_ROWS = 4;   // see launch()

struct Side {   // queries or keys
  const uint16_t *x, *w;
  uint16_t* y;
  long long ld, hd, y_ld, y_hd;
};

struct Params {
  Side q, k;
  const int32_t* positions;
  int n_tokens, h_q, heads, lanes;   // heads: of both; lanes: of a row that hold values
  int rows, q_chunks, chunks;        // heads of a lane group, and lane groups of a token: of its queries, and all
  int first, half;                   // parts of 8 values: the first rotary one, and half of them
  int interleaved, fp16;
  float inv_d, eps;
  // rotary frequency of pair i as a 64-bit fixed-point fraction of a turn
  unsigned long long turns[MAX_PAIRS];
};

template <bool FP16>
__device__ __forceinline__ float2 unpack(uint32_t w) {
  if (FP16) return __half22float2(*reinterpret_cast<const __half2*>(&w));
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
template <bool FP16>
__device__ __forceinline__ uint32_t pack(float2 v) {
  if (FP16) return dsa::pack_f16x2(v.x, v.y);
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(v.y), "f"(v.x));
  return r;
}
template <bool FP16>
__device__ __forceinline__ void unpack8(uint4 v, float2* f) {
  f[0] = unpack<FP16>(v.x);
  f[1] = unpack<FP16>(v.y);
  f[2] = unpack<FP16>(v.z);
  f[3] = unpack<FP16>(v.w);
}
// two fp32 operations in one instruction
__device__ __forceinline__ unsigned long long bits(float2 v) {
  unsigned long long r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(v.x), "f"(v.y));
  return r;
}
__device__ __forceinline__ float2 floats(unsigned long long v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  unsigned long long r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits(a)), "l"(bits(b)));
  return floats(r);
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  unsigned long long r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(bits(a)), "l"(bits(b)), "l"(bits(c)));
  return floats(r);
}

template <int G, bool INTERLEAVED, bool FP16>
__global__ void __launch_bounds__(THREADS) norm_rope_kernel(const __grid_constant__ Params P) {
  const int l = threadIdx.x & (G - 1);
  const long long unit = (long long)blockIdx.x * (THREADS / G) + threadIdx.x / G, at = unit / P.chunks;
  const bool there = at < P.n_tokens;
  const int token = there ? (int)at : P.n_tokens - 1, chunk = (int)(unit - at * P.chunks);
  const bool key = chunk >= P.q_chunks, holds = l < P.lanes;
  // heads of this lane group, all of the queries or all of the keys
  const int head0 = (chunk - (key ? P.q_chunks : 0)) * P.rows, heads = key ? P.heads - P.h_q : P.h_q;
  const int rows = there && holds ? min(P.rows, heads - head0) : 0;
  const uint16_t* w = key ? P.k.w : P.q.w;
  const long long hd = key ? P.k.hd : P.q.hd, y_hd = key ? P.k.y_hd : P.q.y_hd;
  const uint16_t* x_row = (key ? P.k.x : P.q.x) + token * (key ? P.k.ld : P.q.ld) + head0 * hd;
  uint16_t* y_row = (key ? P.k.y : P.q.y) + token * (key ? P.k.y_ld : P.q.y_ld) + head0 * y_hd;

  // this lane's parts of 8 values: parts of a head are numbered 0 .. 2 lanes - 1
  int part[2] = {2 * l, 2 * l + 1};
  bool turns = false;   // both parts turn; else, interleaved, each may
  if (!INTERLEAVED) {
    if (l < P.half) {
      part[0] = P.first + l;
      part[1] = P.first + P.half + l;
      turns = true;
    } else {   // of the parts in front of the rotary ones and behind them
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        part[s] -= 2 * P.half;
        if (part[s] >= P.first) part[s] += 2 * P.half;
      }
    }
  }
  struct Row {
    uint4 v[2];
  };
  auto load = [&](int i) {
    Row r;
    r.v[0] = r.v[1] = make_uint4(0u, 0u, 0u, 0u);
    if (i < rows) {
      const uint16_t* x = x_row + i * hd;
      r.v[0] = *reinterpret_cast<const uint4*>(x + 8 * part[0]);
      r.v[1] = *reinterpret_cast<const uint4*>(x + 8 * part[1]);
    }
    return r;
  };
  const int pos = __ldg(P.positions + token);
  Row v[AT_ONCE];
#pragma unroll
  for (int a = 0; a < AT_ONCE; ++a) v[a] = load(a);
  const bool norm = w != nullptr;
  float2 weight[8];
#pragma unroll
  for (int s = 0; s < 2; ++s)
    unpack8<FP16>(holds && norm ? __ldg(reinterpret_cast<const uint4*>(w) + part[s]) : make_uint4(0u, 0u, 0u, 0u), weight + 4 * s);
  // (cos, sin) of this lane's pairs: of the values e of both parts, or, interleaved, of the pairs of the first part and
  // of the second
  float cs[8], sn[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    int pair = 8 * l + e;
    bool turn = turns;
    if (INTERLEAVED) {
      const int p = part[e >> 2] - P.first;
      turn = p >= 0 && p < 2 * P.half;
      pair = 4 * p + (e & 3);
    }
    cs[e] = 1.f;
    sn[e] = 0.f;
    if (turn) {
      const unsigned long long t = (unsigned long long)(long long)pos * P.turns[pair];
      sincospif((float)(t >> 40) * 1.1920928955078125e-07f, &sn[e], &cs[e]);   // 2 * (its 24 highest bits / 2^24)
    }
  }

  // every lane group of a warp makes the same trips: shuffles
  for (int i0 = 0; i0 < P.rows; i0 += AT_ONCE) {
#pragma unroll
    for (int a = 0; a < AT_ONCE; ++a) {
      const int i = i0 + a;
      if (i >= P.rows) break;
      float2 x[8];
#pragma unroll
      for (int s = 0; s < 2; ++s) unpack8<FP16>(v[a].v[s], x + 4 * s);
      v[a] = load(i + AT_ONCE);
      float2 ss = mul2(x[0], x[0]);
#pragma unroll
      for (int e = 1; e < 8; ++e) ss = fma2(x[e], x[e], ss);
      float sum = ss.x + ss.y;
#pragma unroll
      for (int o = G / 2; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
      if (norm) {
        const float inv = __frsqrt_rn(fmaf(sum, P.inv_d, P.eps));
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = mul2(mul2(x[e], make_float2(inv, inv)), weight[e]);
      }
      // values that do not turn are left as they are: 0 * infinity is not 0
      if (INTERLEAVED) {
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          const int p = part[s] - P.first;
          if (p >= 0 && p < 2 * P.half) {
#pragma unroll
            for (int e = 4 * s; e < 4 * s + 4; ++e)
              x[e] = make_float2(fmaf(x[e].x, cs[e], -x[e].y * sn[e]), fmaf(x[e].x, sn[e], x[e].y * cs[e]));
          }
        }
      } else if (turns) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 c = make_float2(cs[2 * e], cs[2 * e + 1]), n = make_float2(sn[2 * e], sn[2 * e + 1]);
          const float2 b = x[4 + e];
          x[4 + e] = fma2(x[e], n, mul2(b, c));
          x[e] = fma2(x[e], c, mul2(b, make_float2(-n.x, -n.y)));
        }
      }
      if (i < rows) {
        uint16_t* y = y_row + i * y_hd;
#pragma unroll
        for (int s = 0; s < 2; ++s)
          *reinterpret_cast<uint4*>(y + 8 * part[s]) =
              make_uint4(pack<FP16>(x[4 * s]), pack<FP16>(x[4 * s + 1]), pack<FP16>(x[4 * s + 2]), pack<FP16>(x[4 * s + 3]));
      }
    }
  }
}

static bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

static int check(const dsa_qk_params* p) {
  if (!p || p->n_tokens < 0 || p->n_tokens > (1 << 30) || p->h_q < 1 || p->h_k < 0 || p->rotary_dim < 0 || p->rotary_start < 0 ||
      (p->type != DSA_QK_BF16 && p->type != DSA_QK_FP16) || (p->flags & ~DSA_QK_FLAG_INTERLEAVED) != 0 ||
      !(p->rms_eps >= 0.f) || !isfinite(p->rms_eps) || !(p->rope_base > 0.f) || !isfinite(p->rope_base))
    return DSA_ERR_INVALID_ARG;
  if (p->d < 64 || p->d > 256 || p->d % 16 != 0 || p->rotary_dim % 16 != 0 || p->rotary_start % 8 != 0 ||
      p->rotary_dim > p->d || p->rotary_start > p->d - p->rotary_dim || p->h_q > DSA_QK_MAX_HEADS ||
      p->h_k > DSA_QK_MAX_HEADS - p->h_q)
    return DSA_ERR_UNSUPPORTED_SHAPE;
  return DSA_OK;
}

static void turn_table(float base, int dim, unsigned long long* out) {
  // a function of two numbers, kept by each host thread for the last ones: the powers take 5 us
  static thread_local float known_base = 0.f;
  static thread_local int known_dim = -1;
  static thread_local unsigned long long known[MAX_PAIRS];
  if (base != known_base || dim != known_dim) {
    const long double two_pi = 6.283185307179586476925286766559L;
    for (int i = 0; i < dim / 2; ++i) {
      const long double f = powl((long double)base, -2.0L * i / dim) / two_pi;
      known[i] = (unsigned long long)((f - floorl(f)) * 18446744073709551616.0L);
    }
    known_base = base;
    known_dim = dim;
  }
  for (int i = 0; i < dim / 2; ++i) out[i] = known[i];
}

template <int G>
static int launch(const Params& P, int sms, cudaStream_t st) {
  Params Q = P;
  constexpr int groups = THREADS / G;
  // As many rows of a lane group as leave every SM SPREAD CTAs or fewer, and of those the number that costs a
  // token least: groups take as long as the fullest one, and a group's angles as long as some rows.  us, SPREAD
  // 4 and 8: 2123 tokens of 16 heads of 192 10.4 and 14.4; 64 of 64 + 8 of 128 10.5 and 10.7.  (With AT_ONCE 2
  // in place of 4, 16381 of these 118.8 against 104.6.)
  const long long total = (long long)P.n_tokens * P.heads, spread = (long long)SPREAD * sms * groups;
  const long long most = (total + spread - 1) / spread < MOST_ROWS ? (total + spread - 1) / spread : MOST_ROWS;
  long long least = 1LL << 60;
  for (int rows = 1; rows <= most; ++rows) {
    const int q_chunks = (P.h_q + rows - 1) / rows, chunks = q_chunks + (P.heads - P.h_q + rows - 1) / rows;
    const long long cost = (long long)chunks * (rows + ANGLE_ROWS);
    if (cost <= least) {
      least = cost;
      Q.rows = rows;
      Q.q_chunks = q_chunks;
      Q.chunks = chunks;
    }
  }
  const long long grid = ((long long)P.n_tokens * Q.chunks + groups - 1) / groups;
  if (grid > 0x7FFFFFFFLL) return DSA_ERR_UNSUPPORTED_SHAPE;
  auto run = [&](auto kernel) { kernel<<<(unsigned)grid, THREADS, 0, st>>>(Q); };
  if (P.fp16) P.interleaved ? run(norm_rope_kernel<G, true, true>) : run(norm_rope_kernel<G, false, true>);
  else P.interleaved ? run(norm_rope_kernel<G, true, false>) : run(norm_rope_kernel<G, false, false>);
  return cudaGetLastError() == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}

}  // namespace dsa_qk

extern "C" int dsa_qk_params_init(dsa_qk_params* p, int32_t n_tokens, int32_t h_q, int32_t h_k, int32_t d) {
  if (!p) return DSA_ERR_INVALID_ARG;
  p->n_tokens = n_tokens;
  p->h_q = h_q;
  p->h_k = h_k;
  p->d = d;
  p->rotary_dim = d;
  p->rotary_start = 0;
  p->type = DSA_QK_BF16;
  p->flags = 0;
  p->rms_eps = 1e-6f;
  p->rope_base = 10000.0f;
  return dsa_qk::check(p);
}

extern "C" int dsa_qk_norm_rope(const void* q, int64_t q_ld, int64_t q_hd, const void* k, int64_t k_ld, int64_t k_hd,
                                const int32_t* positions, const void* q_w, const void* k_w, void* q_out, int64_t q_out_ld,
                                int64_t q_out_hd, void* k_out, int64_t k_out_ld, int64_t k_out_hd, const dsa_qk_params* p,
                                void* stream) {
  using namespace dsa_qk;
  const int rc = check(p);
  if (rc != DSA_OK) return rc;
  if (p->n_tokens == 0) return DSA_OK;
  auto bad_side = [&](const void* x, int64_t ld, int64_t hd, int h) {
    return !x || !aligned(x, 16) || ld % 8 != 0 || hd % 8 != 0 || ld < 0 || hd < 0 || (p->n_tokens > 1 && ld < p->d) ||
           (h > 1 && hd < p->d);
  };
  if (bad_side(q, q_ld, q_hd, p->h_q) || bad_side(q_out, q_out_ld, q_out_hd, p->h_q) || !aligned(q_w, 16))
    return DSA_ERR_INVALID_ARG;
  if (p->h_k > 0 && (bad_side(k, k_ld, k_hd, p->h_k) || bad_side(k_out, k_out_ld, k_out_hd, p->h_k) || !aligned(k_w, 16)))
    return DSA_ERR_INVALID_ARG;
  if ((q_out == q && (q_out_ld != q_ld || q_out_hd != q_hd)) || (p->h_k > 0 && k_out == k && (k_out_ld != k_ld || k_out_hd != k_hd)))
    return DSA_ERR_INVALID_ARG;
  if (!positions || !aligned(positions, 4)) return DSA_ERR_INVALID_ARG;
  int sms = 0;
  const int device_rc = dsa::gb300_sms(&sms);
  if (device_rc != DSA_OK) return device_rc;
  Params P;
  auto side = [](const void* x, int64_t ld, int64_t hd, const void* w, void* y, int64_t y_ld, int64_t y_hd) {
    return Side{static_cast<const uint16_t*>(x), static_cast<const uint16_t*>(w), static_cast<uint16_t*>(y), (long long)ld,
                (long long)hd, (long long)y_ld, (long long)y_hd};
  };
  P.q = side(q, q_ld, q_hd, q_w, q_out, q_out_ld, q_out_hd);
  P.k = p->h_k > 0 ? side(k, k_ld, k_hd, k_w, k_out, k_out_ld, k_out_hd) : Side{};
  P.positions = positions;
  P.n_tokens = p->n_tokens;
  P.h_q = p->h_q;
  P.heads = p->h_q + p->h_k;
  P.lanes = p->d / 16;
  P.rows = P.q_chunks = P.chunks = 0;
  P.first = p->rotary_start / 8;
  P.half = p->rotary_dim / 16;
  P.interleaved = (p->flags & DSA_QK_FLAG_INTERLEAVED) != 0;
  P.fp16 = p->type == DSA_QK_FP16;
  P.inv_d = 1.0f / (float)p->d;
  P.eps = p->rms_eps;
  turn_table(p->rope_base, p->rotary_dim, P.turns);
  const cudaStream_t st = (cudaStream_t)stream;
  return p->d <= 64 ? launch<4>(P, sms, st) : p->d <= 128 ? launch<8>(P, sms, st) : launch<16>(P, sms, st);
}
