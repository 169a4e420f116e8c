// Insert into the paged 8-bit cache (include/dsa_kv8.h): new tokens' keys and values as
// E4M3 codes under one power-of-two scale per page and KV head.
//
// A CTA takes the runs (new tokens of one page) that start in its window of the batch, for
// some of the pairs (KV head, keys or values); a run that passes the window's end is
// finished by the CTA where it starts, so no two CTAs touch one page of a pair.  The runs
// are found once.  D / 8 lanes hold a token (16 bytes each), so that a row is read in one
// piece.  For each pair:
//   1. every token of the CTA's runs is read once into registers, and its largest
//      magnitude goes into its run's maximum (shared memory, an integer maximum of the
//      bits, which order as the magnitudes do);
//   2. one thread per run forms the scale from the maximum's exponent, writes it, and
//      lists the run if the page's older rows have to be rescaled;
//   3. the registers are scaled, rounded and written; then the listed runs' older rows.
// Bound by memory: 2 bytes read and 1 written per value; the older rows are read only
// where a page's scale grows, which a new token does less and less often as a page fills.
// 67 k tokens, 8 heads of 128: 412 MB in 77 us, 5.4 TB/s, 0.79 of a copy's rate.  (It was
// bound by instruction issue, 76 %, until the lanes of a warp took neighbouring
// tokens, maxima were taken two values at a time and the windows filled the CTA.)

#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>
#include <type_traits>

#include "dsa_kv8.h"
#include "ptx_sm103.cuh"

namespace dsa_kv8_insert_impl {

constexpr int THREADS = 256;
constexpr int CTAS = 152 * 4;   // about what a GB300 holds at once
constexpr uint32_t NONE = 0xFFFFFFFFu;
constexpr int WINDOW = 112;  // most tokens in which a CTA's runs start

struct Params {
  const uint16_t *x[2];
  long long ld[2], hd[2];
  uint8_t* pool[2];
  float* scale[2];
  const int64_t* slots;
  uint32_t* status;
  long long n_rows;
  int n_tokens, h_kv, page_shift, window;
  int pairs, splits;   // (head, keys or values) pairs of a CTA, CTAs of a window
};

template <bool FP16>
__device__ __forceinline__ float2 to_f32x2(uint32_t w) {
  if (FP16) return __half22float2(*reinterpret_cast<const __half2*>(&w));
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
// larger of two values each, by lane of the word; a NaN loses
template <bool FP16>
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
  uint32_t r;
  if (FP16) asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  else asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Magnitudes of two values, a NaN for an infinity: |x| * 0 + |x|.  An infinity in the maximum would
// take its whole page to zero.  (Looking for one behind the maximum, and taking that once more, cost
// registers: 67 k tokens 77 to 84 us, against 76.4 so and 75.5 without.)
template <bool FP16>
__device__ __forceinline__ uint32_t magnitudes(uint32_t w) {
  uint32_t r;
  if (FP16) asm("{\n\t.reg .b32 a;\n\tabs.f16x2 a, %1;\n\tfma.rn.f16x2 %0, a, %2, a;\n\t}" : "=r"(r) : "r"(w), "r"(0u));
  else asm("{\n\t.reg .b32 a;\n\tabs.bf16x2 a, %1;\n\tfma.rn.bf16x2 %0, a, %2, a;\n\t}" : "=r"(r) : "r"(w), "r"(0u));
  return r;
}

// E4M3 codes of f * s (two products in one instruction)
__device__ __forceinline__ uint32_t scaled_codes(float2 f, float s) {
  uint64_t v, m;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(f.x), "f"(f.y));
  asm("mov.b64 %0, {%1, %1};" : "=l"(m) : "f"(s));
  asm("mul.rn.f32x2 %0, %0, %1;" : "+l"(v) : "l"(m));
  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
  return dsa::f32x2_to_e4m3x2(f.x, f.y);
}

// least power of two s >= 2^-64 with amax <= 448 s = 1.75 * 2^8 s, at most 2^64
__device__ __forceinline__ float page_scale(uint32_t amax_bits) {
  int e = (int)(amax_bits >> 23) - 127 - 8;
  if ((amax_bits & 0x7FFFFFu) > 0x600000u) ++e;
  e = min(max(e, -64), 64);
  return __uint_as_float((uint32_t)(e + 127) << 23);
}

template <int D, int PASSES, bool FP16>
__global__ void __launch_bounds__(THREADS, PASSES * D <= 1024 ? 4 : 2) insert_kernel(const __grid_constant__ Params P) {
  constexpr int LANES = D / 8;                    // lanes of one token
  constexpr int GROUPS = THREADS / LANES;         // tokens per pass
  constexpr int SPAN = PASSES * GROUPS;           // tokens that the CTA may hold
  __shared__ long long s_slot[SPAN + 1];          // [i + 1]: slot of token t0 + i
  // a token's row in the pool's first head and the first token of its run; NONE: not this CTA's
  __shared__ uint2 s_to[SPAN];
  __shared__ uint32_t s_amax[2][WINDOW];          // by the run's first token, of this pair and the next
  __shared__ float s_scale[WINDOW];               // 1 / scale
  __shared__ int s_last[THREADS / 32];
  __shared__ int s_n_old[2], s_old_end[WINDOW], s_old_run[WINDOW];
  __shared__ float s_old_ratio[WINDOW];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int t0 = blockIdx.x / P.splits * P.window;
  const int pairs = 2 * P.h_kv;
  const int pair0 = blockIdx.x % P.splits * P.pairs, pair1 = min(pair0 + P.pairs, pairs);
  const int page_mask = (1 << P.page_shift) - 1;
  static_assert(SPAN <= THREADS, "one thread per token");

  // ---- the window's runs
  long long slot = -1;
  if (tid < SPAN && t0 + tid < P.n_tokens) {
    slot = P.slots[t0 + tid];
    if (slot >= P.n_rows) {
      if (pair0 == 0 && P.status) atomicOr(P.status, DSA_STATUS_SLOT_OUT_OF_RANGE);
      slot = -1;
    }
  }
  if (tid < SPAN) s_slot[tid + 1] = slot;
  if (tid == 0) {
    const long long before = t0 > 0 ? P.slots[t0 - 1] : -1;
    s_slot[0] = before >= P.n_rows ? -1 : before;
    s_n_old[0] = 0;
  }
  if (tid < WINDOW) s_amax[0][tid] = 0u;
  __syncthreads();
  const bool starts = slot >= 0 && ((slot & page_mask) == 0 || s_slot[tid] != slot - 1);
  // the last start or gap at or before each token
  const uint32_t breaks = __ballot_sync(0xFFFFFFFFu, slot < 0 || starts);
  const uint32_t upto = breaks & (0xFFFFFFFFu >> (31 - lane));
  int from = upto ? 32 * w + 31 - __clz(upto) : -1;
  if (lane == 31) s_last[w] = from;
  __syncthreads();
  for (int u = w - 1; u >= 0 && from < 0; --u) from = s_last[u];
  // `from` is the run's start if a run starts there: -1 (the run began before this window)
  // and starts past the window belong to another CTA
  if (tid < SPAN) {
    const uint32_t row = ((uint32_t)(slot >> P.page_shift) * P.h_kv << P.page_shift) + ((uint32_t)slot & page_mask);
    s_to[tid] = (slot >= 0 && from >= 0 && from < P.window) ? make_uint2(row, (uint32_t)from) : make_uint2(NONE, NONE);
  }
  const bool own = tid < P.window && starts, continues = own && (slot & page_mask) != 0;
  __syncthreads();

  const int group = tid / LANES, part = tid % LANES;
  for (int pair = pair0; pair < pair1; ++pair) {
    const int which = pair >= P.h_kv ? 1 : 0, head = which ? pair - P.h_kv : pair;
    const int now = (pair - pair0) & 1;
    // ---- 1. values into registers, maxima of the runs
    const uint16_t* const src = P.x[which] + head * P.hd[which] + part * 8;
    const long long ld = P.ld[which];
    uint4 x[PASSES];
    uint2 to[PASSES];
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
      const int i = group * PASSES + p;   // neighbours, so that a lane joins the maxima of a run's tokens
      to[p] = s_to[i];
      x[p] = make_uint4(0u, 0u, 0u, 0u);
      if (to[p].x != NONE) x[p] = dsa::ldg_nc(src + (t0 + i) * ld);
    }
    float* const scale_at = P.scale[which] + (slot >> P.page_shift) * P.h_kv + head;
    float old = 0.f;
    if (continues) old = *scale_at;
    uint32_t m2 = 0u;   // of the tokens since the last run's end
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
      m2 = max2<FP16>(m2, max2<FP16>(max2<FP16>(magnitudes<FP16>(x[p].x), magnitudes<FP16>(x[p].y)),
                                     max2<FP16>(magnitudes<FP16>(x[p].z), magnitudes<FP16>(x[p].w))));
      // on to the next token, unless a run of the warp's ends here
      if (p + 1 < PASSES && __all_sync(0xFFFFFFFFu, to[p + 1 < PASSES ? p + 1 : p].y == to[p].y)) continue;
      const bool some = to[p].x != NONE;
      if (__any_sync(0xFFFFFFFFu, some)) {
#pragma unroll
        for (int o = LANES / 2; o >= 1; o >>= 1) m2 = max2<FP16>(m2, __shfl_xor_sync(0xFFFFFFFFu, m2, o));
        const float2 m = to_f32x2<FP16>(m2);
        // fmaxf leaves out a NaN (which is all that was there, if it is still here)
        if (part == 0 && some) atomicMax(&s_amax[now][to[p].y], __float_as_uint(fmaxf(0.f, fmaxf(m.x, m.y))));
      }
      m2 = 0u;
    }
    __syncthreads();

    // ---- 2. scales
    if (own) {
      float s = page_scale(s_amax[now][tid]);
      if (continues) {
        if (old >= s) {
          s = old;
        } else {
          const int k = atomicAdd(&s_n_old[now], 1);   // the order of the list changes no result
          s_old_run[k] = tid;
          s_old_ratio[k] = old / s;
        }
      }
      *scale_at = s;
      s_scale[tid] = 1.0f / s;
    }
    if (tid < WINDOW) s_amax[now ^ 1][tid] = 0u;
    if (tid == 0) s_n_old[now ^ 1] = 0;
    __syncthreads();

    // ---- 3. codes
    uint8_t* const dst = P.pool[which] + part * 8;
    const uint32_t head_rows = (uint32_t)head << P.page_shift;
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
      if (to[p].x == NONE) continue;
      const float inv = s_scale[to[p].y];
      const uint32_t v[4] = {x[p].x, x[p].y, x[p].z, x[p].w};
      uint32_t c[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 f = to_f32x2<FP16>(v[k]);
        c[k] = scaled_codes(f, inv);
      }
      *reinterpret_cast<uint2*>(dst + (uint64_t)(to[p].x + head_rows) * D) = make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
    }

    // the older rows of pages whose scale grew: (run, row) pairs over the groups
    const int n_old = s_n_old[now];
    if (n_old == 0) continue;
    if (tid == 0) {
      int sum = 0;
      for (int k = 0; k < n_old; ++k) {
        sum += (int)s_slot[s_old_run[k] + 1] & page_mask;
        s_old_end[k] = sum;
      }
    }
    __syncthreads();
    const int rows = s_old_end[n_old - 1];
    for (int f = group; f < rows; f += GROUPS) {
      int k = 0;
      while (s_old_end[k] <= f) ++k;
      const int r = f - (k > 0 ? s_old_end[k - 1] : 0);
      const float ratio = s_old_ratio[k];
      const uint32_t page = (uint32_t)(s_slot[s_old_run[k] + 1] >> P.page_shift);
      const uint32_t row = ((page * P.h_kv + head) << P.page_shift) + r;
      uint2* const at = reinterpret_cast<uint2*>(dst + (uint64_t)row * D);
      const uint2 c = *at;
      const uint32_t in[4] = {c.x & 0xFFFFu, c.x >> 16, c.y & 0xFFFFu, c.y >> 16};
      uint32_t o[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t h2 = dsa::e4m3x2_to_f16x2(in[e]);
        const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&h2));
        o[e] = dsa::f32x2_to_e4m3x2(v.x * ratio, v.y * ratio);
      }
      *at = make_uint2(o[0] | (o[1] << 16), o[2] | (o[3] << 16));
    }
  }
}

static bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

static bool bad_pitch(int64_t ld, int64_t hd, int heads, int d) {
  return ld < d || ld % 8 != 0 || hd % 8 != 0 || (heads > 1 && hd < d);
}

}  // namespace dsa_kv8_insert_impl

extern "C" int dsa_kv8_insert(const void* k, int64_t k_ld, int64_t k_hd, const void* v, int64_t v_ld, int64_t v_hd,
                              const int64_t* slots, int32_t n_tokens, int32_t type, void* k_pool, void* v_pool,
                              float* k_scale, float* v_scale, int32_t n_pages, int32_t h_kv, int32_t page_size,
                              int32_t d, uint32_t* status, void* stream) {
  using namespace dsa_kv8_insert_impl;
  if (n_tokens < 0 || n_tokens > (1 << 30) || n_pages < 0 || h_kv < 1 || (type != DSA_KV8_BF16 && type != DSA_KV8_FP16))
    return DSA_ERR_INVALID_ARG;
  if ((d != 64 && d != 128) || (page_size != 16 && page_size != 32 && page_size != 64 && page_size != 128) ||
      h_kv > DSA_KV8_MAX_HEADS || (long long)n_pages * h_kv * page_size >= (1LL << 32) - 1)   // rows are numbered in 32 bits
    return DSA_ERR_UNSUPPORTED_SHAPE;
  if (n_tokens == 0) return DSA_OK;
  if (bad_pitch(k_ld, k_hd, h_kv, d) || bad_pitch(v_ld, v_hd, h_kv, d)) return DSA_ERR_INVALID_ARG;
  if (!k || !v || !slots || !aligned(k, 16) || !aligned(v, 16) || !aligned(slots, 8) || (status && !aligned(status, 4)))
    return DSA_ERR_INVALID_ARG;
  if (n_pages > 0 && (!k_pool || !v_pool || !k_scale || !v_scale)) return DSA_ERR_INVALID_ARG;
  if (!aligned(k_pool, 16) || !aligned(v_pool, 16) || !aligned(k_scale, 4) || !aligned(v_scale, 4))
    return DSA_ERR_INVALID_ARG;
  int dev = 0, major = 0, minor = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return DSA_ERR_CUDA;
  cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev);
  cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev);
  if (major != 10 || minor != 3) return DSA_ERR_UNSUPPORTED_DEVICE;
  Params P;
  P.x[0] = static_cast<const uint16_t*>(k);
  P.x[1] = static_cast<const uint16_t*>(v);
  P.ld[0] = k_ld;
  P.ld[1] = v_ld;
  P.hd[0] = k_hd;
  P.hd[1] = v_hd;
  P.pool[0] = static_cast<uint8_t*>(k_pool);
  P.pool[1] = static_cast<uint8_t*>(v_pool);
  P.scale[0] = k_scale;
  P.scale[1] = v_scale;
  P.slots = slots;
  P.status = status;
  P.n_rows = (long long)n_pages * page_size;
  P.n_tokens = n_tokens;
  P.h_kv = h_kv;
  P.page_shift = __builtin_ctz(page_size);
  // the last run of a window may have page_size - 1 more tokens: with them a CTA holds 128
  // tokens, or 192 for pages of 128
  P.window = (page_size > 64 ? 192 : 128) - page_size;
  // as many pairs to a CTA, which finds its runs once, as leave four rounds of CTAs
  const long long windows = (n_tokens + P.window - 1) / P.window;
  const long long rounds = windows * h_kv * 2 / (4LL * CTAS);
  P.pairs = (int)(rounds < 1 ? 1 : rounds > 8 ? 8 : rounds);
  P.splits = (2 * h_kv + P.pairs - 1) / P.pairs;
  if (windows * P.splits >= (1LL << 31)) return DSA_ERR_UNSUPPORTED_SHAPE;
  const unsigned grid = (unsigned)(windows * P.splits);
  cudaStream_t st = (cudaStream_t)stream;
  const bool wide = page_size > 64;
  auto launch = [&](auto fp16) {
    constexpr bool F = decltype(fp16)::value;
    if (d == 128) {
      if (!wide) insert_kernel<128, 8, F><<<grid, THREADS, 0, st>>>(P);
      else insert_kernel<128, 12, F><<<grid, THREADS, 0, st>>>(P);
    } else {
      if (!wide) insert_kernel<64, 4, F><<<grid, THREADS, 0, st>>>(P);
      else insert_kernel<64, 6, F><<<grid, THREADS, 0, st>>>(P);
    }
  };
  if (type == DSA_KV8_FP16) launch(std::true_type());
  else launch(std::false_type());
  return cudaGetLastError() == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}
