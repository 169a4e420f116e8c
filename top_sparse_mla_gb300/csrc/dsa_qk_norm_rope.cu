// RMS norm and rotation of the heads of queries and keys (include/dsa_qk_norm_rope.h).
//
// What bounds it: memory, each value read and written once.  The rows (token, head) of q and
// k are numbered token by token, and a CTA has R neighbouring ones.  It forms the cosines and
// sines of its tokens once, in shared memory, for all their heads, while its first rows are on
// their way.  A row belongs to G lanes of 8 values each (16-byte loads and stores).  Halves of
// a head that turn together lie rotary_dim / 16 lanes apart and are exchanged by shuffles.
//
// The angle of pair i is position * turns[i] in 64-bit fixed point, a fraction of a turn that
// wraps by itself: an fp32 angle would be off by 2^-24 of itself, half a turn at position 2^24.

#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "dsa_qk_norm_rope.h"
#include "ptx_sm103.cuh"

namespace dsa_qk {

constexpr int THREADS = 256;
constexpr int MAX_PAIRS = 128;     // rotary pairs of a head
constexpr int TABLE = 4096;        // cosines and sines of a CTA: 32 KB
constexpr int AT_ONCE = 4;         // rows of a lane group in flight

struct Side {   // queries or keys
  const uint16_t *x, *w;
  uint16_t* y;
  long long ld, hd, y_ld, y_hd;
};

struct Params {
  Side q, k;
  const int32_t* positions;
  int n_tokens, h_q, heads, lanes;   // heads: of both; lanes: of a row that hold values
  int rows;                          // of a CTA
  int pairs, first, half;            // rotary pairs; first lane of the rotary values; lanes of half of them
  int interleaved, fp16;
  float inv_d, eps;
  // rotary frequency of pair i as a 64-bit fixed-point fraction of a turn
  unsigned long long turns[MAX_PAIRS];
};

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
__device__ __forceinline__ void unpack8(uint4 v, int fp16, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 p = unpack(w[i], fp16);
    f[2 * i] = p.x;
    f[2 * i + 1] = p.y;
  }
}

template <int G, bool INTERLEAVED>
__global__ void __launch_bounds__(THREADS) norm_rope_kernel(const __grid_constant__ Params P) {
  extern __shared__ __align__(16) float2 table[];   // [tokens of the CTA][pairs] (cos, sin)
  constexpr int GROUPS = THREADS / G;
  const int lane = threadIdx.x & 31, l = lane & (G - 1), group = threadIdx.x / G;
  const long long row0 = (long long)blockIdx.x * P.rows;
  const long long token0 = row0 / P.heads;
  const int head0 = (int)(row0 - token0 * P.heads);
  const int rows = (int)min((long long)P.rows, (long long)P.n_tokens * P.heads - row0);
  const int fp16 = P.fp16;
  const bool holds = l < P.lanes;

  struct Row {
    int token, head;   // counted from token0
  };
  auto row = [&](int i) {
    const unsigned at = (unsigned)(head0 + i);
    const unsigned t = at / (unsigned)P.heads;
    return Row{(int)t, (int)(at - t * P.heads)};
  };
  auto load = [&](int i) -> uint4 {
    if (i >= rows || !holds) return make_uint4(0u, 0u, 0u, 0u);
    const Row r = row(i);
    const bool key = r.head >= P.h_q;
    const Side& s = key ? P.k : P.q;
    return *reinterpret_cast<const uint4*>(s.x + (token0 + r.token) * s.ld + (r.head - (key ? P.h_q : 0)) * s.hd + 8 * l);
  };

  uint4 v[AT_ONCE];
#pragma unroll
  for (int a = 0; a < AT_ONCE; ++a) v[a] = load(group + a * GROUPS);

  const int tokens = row(rows - 1).token + 1;
  for (int i = threadIdx.x; i < tokens * P.pairs; i += THREADS) {
    const int t = i / P.pairs, pair = i - t * P.pairs;
    const unsigned long long turn = (unsigned long long)(long long)__ldg(P.positions + token0 + t) * P.turns[pair];
    float sn, cs;
    sincospif((float)(turn >> 40) * 1.1920928955078125e-07f, &sn, &cs);   // 2 * (its 24 highest bits / 2^24)
    table[i] = make_float2(cs, sn);
  }
  uint4 qw = make_uint4(0u, 0u, 0u, 0u), kw = qw;
  if (holds && P.q.w) qw = __ldg(reinterpret_cast<const uint4*>(P.q.w) + l);
  if (holds && P.k.w) kw = __ldg(reinterpret_cast<const uint4*>(P.k.w) + l);
  __syncthreads();

  // this lane's place among the rotary values
  const int at = l - P.first;
  const bool turns = at >= 0 && at < 2 * P.half;
  const int partner = (lane & ~(G - 1)) + (turns ? (at < P.half ? l + P.half : l - P.half) : l);
  const int pair0 = INTERLEAVED ? 4 * at : 8 * (at < P.half ? at : at - P.half);
  const float side = at < P.half ? -1.f : 1.f;

  for (int i0 = group; i0 < rows + group; i0 += AT_ONCE * GROUPS) {   // the same trips for every group: shuffles
#pragma unroll
    for (int a = 0; a < AT_ONCE; ++a) {
      const int i = i0 + a * GROUPS;
      const bool live = i < rows;
      const Row r = row(min(i, rows - 1));
      const bool key = r.head >= P.h_q;
      float x[8];
      unpack8(v[a], fp16, x);
      v[a] = load(i + AT_ONCE * GROUPS);
      const bool norm = (key ? P.k.w : P.q.w) != nullptr;
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
      for (int o = G / 2; o >= 1; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
      if (norm) {
        const float inv = 1.0f / sqrtf(fmaf(ss, P.inv_d, P.eps));
        float w[8];
        unpack8(key ? kw : qw, fp16, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = x[e] * inv * w[e];
      }
      const float2* cs = table + (turns ? r.token * P.pairs + pair0 : 0);
      if (INTERLEAVED) {
        if (turns) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 f = cs[e];
            const float b = x[2 * e + 1];
            x[2 * e + 1] = fmaf(x[2 * e], f.y, b * f.x);
            x[2 * e] = fmaf(x[2 * e], f.x, -b * f.y);
          }
        }
      } else if (P.pairs > 0) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float other = __shfl_sync(0xFFFFFFFFu, x[e], partner);
          if (turns) {
            const float2 f = cs[e];
            x[e] = fmaf(x[e], f.x, side * other * f.y);
          }
        }
      }
      if (live && holds) {
        const Side& s = key ? P.k : P.q;
        uint4 o;
        o.x = pack(x[0], x[1], fp16);
        o.y = pack(x[2], x[3], fp16);
        o.z = pack(x[4], x[5], fp16);
        o.w = pack(x[6], x[7], fp16);
        *reinterpret_cast<uint4*>(s.y + (token0 + r.token) * s.y_ld + (r.head - (key ? P.h_q : 0)) * s.y_hd + 8 * l) = o;
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
static int launch(const Params& P, long long total, int sms, cudaStream_t st) {
  Params Q = P;
  constexpr int groups = THREADS / G;
  // as many rows as give every SM its CTAs, at most what AT_ONCE loads of every group bring at
  // four rounds, and no more tokens than the table has room for
  long long rows = (total + 4LL * sms - 1) / (4LL * sms);
  const long long most = 4LL * AT_ONCE * groups;
  if (rows > most) rows = most;
  rows = (rows + groups - 1) / groups * groups;
  // rows that begin anywhere touch at most (rows - 2) / heads + 2 tokens
  const long long tokens = P.pairs > 0 ? TABLE / P.pairs : rows + 1;
  if ((rows - 2) / P.heads + 2 > tokens) rows = (tokens - 2) * P.heads + 1;
  Q.rows = (int)rows;
  const long long grid = (total + rows - 1) / rows;
  if (grid > 0x7FFFFFFFLL) return DSA_ERR_UNSUPPORTED_SHAPE;
  const size_t smem = (size_t)((rows - 2) / P.heads + 2) * P.pairs * sizeof(float2);
  if (P.interleaved) norm_rope_kernel<G, true><<<(unsigned)grid, THREADS, smem, st>>>(Q);
  else norm_rope_kernel<G, false><<<(unsigned)grid, THREADS, smem, st>>>(Q);
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
  int dev = 0, major = 0, minor = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return DSA_ERR_CUDA;
  cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev);
  cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev);
  if (major != 10 || minor != 3) return DSA_ERR_UNSUPPORTED_DEVICE;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return DSA_ERR_CUDA;
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
  P.lanes = p->d / 8;
  P.rows = 0;
  P.pairs = p->rotary_dim / 2;
  P.first = p->rotary_start / 8;
  P.half = p->rotary_dim / 16;
  P.interleaved = (p->flags & DSA_QK_FLAG_INTERLEAVED) != 0;
  P.fp16 = p->type == DSA_QK_FP16;
  P.inv_d = 1.0f / (float)p->d;
  P.eps = p->rms_eps;
  turn_table(p->rope_base, p->rotary_dim, P.turns);
  const long long total = (long long)p->n_tokens * P.heads;
  const cudaStream_t st = (cudaStream_t)stream;
  return p->d <= 64 ? launch<8>(P, total, sms, st) : p->d <= 128 ? launch<16>(P, total, sms, st) : launch<32>(P, total, sms, st);
}
