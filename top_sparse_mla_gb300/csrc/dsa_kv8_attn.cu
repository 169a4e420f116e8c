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

#include <float.h>

#include "dsa_kv8.cuh"

namespace dsa_kv8 {

constexpr int MAX_ROWS = 32;      // most query rows of a request in rows_kernel
constexpr int ROW_WARPS = 4;      // warps of a rows_kernel CTA
constexpr int UNIT_STEPS = 2;     // what a unit (request, KV head) costs a CTA beside its steps, in steps of every warp
constexpr int MIN_STEPS = 2;      // the fewest steps of a warp that are worth a unit's beginning
constexpr int PLAN_THREADS = 1024;
// Requests that a thread of rows_kernel looks at for its CTA's share, at most.  Up to 300
// tokens, 16/2 heads, us, own shares and the plan's: 500 requests 19.9 and 23.5, 1024 32.7
// and 35.4, 1500 47.4 and 50.8, 2048 (16 a thread) 63.3 and 63.6, 4096 124.7 and 111.3.
constexpr int OWN_PLAN = 12;
constexpr int FEW_THREADS = 256;  // of the plan, where rows_kernel's CTAs find their shares
// rows_kernel's CTAs per SM, by head dimension and tiles of 8 query rows: what its registers leave room for.
// Every CTA has to be resident at once, since the plan gives each an equal share.
constexpr int ctas_per_sm(int d, int nt) { return (nt == 1 ? 4 : nt == 2 ? 3 : 2) + (d == 64 ? (nt == 1 ? 2 : 1) : 0); }
constexpr float M_INIT = -FLT_MAX;   // below every score, and finite: 2^(-inf - M_INIT) is 0

// the steps of each of a request's units with what a unit costs beside them; 0 for a
// request that is not rows_kernel's
__device__ __forceinline__ int unit_steps(const Params& P, const Request& a) {
  const bool ours = a.q_len > 0 && a.q_len <= P.max_q_len && a.rows(P) <= P.small_rows;
  return ours ? P.unit_steps + span(P, a, 0, a.q_len - 1).steps : 0;
}
__device__ __forceinline__ long long share_of(const Params& P, long long total) {
  return max((total + P.n_shares - 1) / P.n_shares, (long long)P.min_share);
}
// where among its units the share with `rest` steps of request r in front of it begins
__device__ __forceinline__ Share share_at(const Params& P, int r, long long rest, long long steps) {
  Share s;
  s.req = r;
  s.head = (int)(rest / steps);
  s.step = rest - s.head * steps - P.unit_steps;
  return s;
}

// ------------------------------------------------------------------------------ plan
// The steps of the small requests, all heads of all requests in a row and P.unit_steps more
// in front of each unit's for its beginning and end, are cut into equal shares, one for
// each CTA: a share may begin and end inside a unit, and the CTAs are done at the same time
// whatever the lengths.  The tiles of the other requests are listed.
//
// Of few requests (P.own_plan) every CTA of rows_kernel finds its share for itself while
// this kernel, for the counters and the tiles, is still on its way.
template <int THREADS>
__global__ void __launch_bounds__(THREADS) plan_kernel(const __grid_constant__ Params P) {
  extern __shared__ long long s_step[];   // [n_req + 1] exclusive prefix of the steps
  long long* s_tile = s_step + P.n_req + 1;   // [n_req + 1] of the tiles
  __shared__ long long s_step_warp[THREADS / 32], s_tile_warp[THREADS / 32];
  __shared__ int s_place[THREADS];
  __shared__ uint32_t s_bad;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5, n = P.n_req;
  if (tid == 0) s_bad = 0;
  for (int b = tid; b < 3 * P.n_shares; b += THREADS) P.arrived[b] = 0;
  __syncthreads();
  if (P.own_plan && !P.has_tiles) {   // no shares and no tiles to find
    for (int r = tid; r < n; r += THREADS)
      if (request(P, r).q_len > P.max_q_len) atomicOr(&s_bad, DSA_STATUS_QUERY_TOO_LONG);
    __syncthreads();
    if (tid == 0) {
      P.header->status = s_bad;
      P.header->n_tiles = 0;
    }
    return;
  }
  for (int r = tid; r < n; r += THREADS) {
    const Request a = request(P, r);
    const int rows = a.rows(P);
    int tiles = 0;
    if (a.q_len > P.max_q_len) atomicOr(&s_bad, DSA_STATUS_QUERY_TOO_LONG);
    else if (rows > P.small_rows) tiles = (rows + TILE_ROWS - 1) / TILE_ROWS;
    s_step[r] = unit_steps(P, a);
    s_tile[r] = tiles;
  }
  __syncthreads();
  const int per = ((n + THREADS - 1) / THREADS) | 1;   // odd: no bank conflicts
  const int r0 = min(tid * per, n), r1 = min(r0 + per, n);
  long long st = 0, ti = 0;
  for (int r = r0; r < r1; ++r) {
    st += s_step[r];
    ti += s_tile[r];
  }
  long long st_in = st, ti_in = ti;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long a = __shfl_up_sync(0xFFFFFFFFu, st_in, o), b = __shfl_up_sync(0xFFFFFFFFu, ti_in, o);
    if (lane >= o) {
      st_in += a;
      ti_in += b;
    }
  }
  if (lane == 31) {
    s_step_warp[w] = st_in;
    s_tile_warp[w] = ti_in;
  }
  __syncthreads();
  long long st_ex = st_in - st, ti_ex = ti_in - ti, all = 0, all_tiles = 0;
#pragma unroll
  for (int u = 0; u < THREADS / 32; ++u) {
    if (u < w) {
      st_ex += s_step_warp[u];
      ti_ex += s_tile_warp[u];
    }
    all += s_step_warp[u];
    all_tiles += s_tile_warp[u];
  }
  for (int r = r0; r < r1; ++r) {
    const long long a = s_step[r], b = s_tile[r];
    s_step[r] = st_ex;
    s_tile[r] = ti_ex;
    st_ex += a;
    ti_ex += b;
  }
  if (tid == 0) {
    s_step[n] = all;
    s_tile[n] = all_tiles;
  }
  __syncthreads();

  const long long total = all * P.h_kv;
  const long long share = share_of(P, total);
  // few requests: the CTAs find them for themselves
  for (int b = tid; b < (P.own_plan ? 0 : P.n_shares); b += THREADS) {
    Share s{-1, 0, 0};
    const long long f = b * share;
    if (f < total) {
      int lo = 0, hi = n;   // the request with s_step[lo] * h_kv <= f < s_step[lo + 1] * h_kv
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s_step[mid] * P.h_kv <= f) lo = mid; else hi = mid;
      }
      s = share_at(P, lo, f - s_step[lo] * P.h_kv, s_step[lo + 1] - s_step[lo]);
    }
    P.shares[b] = s;
  }
  // ascending cu_q cannot give more tiles than the list has room for
  const int n_tiles = (int)min(all_tiles, (long long)P.max_tiles);
  if (n_tiles > 0) {
    // the longest first (by cached tokens in blocks of 128, all above THREADS - 1 alike): a count
    // of each length, the places behind the longer ones, then the tiles.  The order among
    // equal ones changes no result.
    auto tile = [&](int i) {
      int lo = 0, hi = n;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s_tile[mid] <= i) lo = mid; else hi = mid;
      }
      const Request a = request(P, lo);
      const int row0 = (int)(i - s_tile[lo]) * TILE_ROWS, row1 = min(row0 + TILE_ROWS, a.rows(P)) - 1;
      Tile t;
      t.req = lo;
      t.row0 = row0;
      t.q0 = a.q0;
      t.rows = a.rows(P);
      t.pos0 = a.kv - a.q_len;
      t.lo = span(P, a, row0 / P.group, row1 / P.group).lo;
      t.hi = max(t.pos0 + row1 / P.group + 1, 0);
      t.pad = 0;
      return t;
    };
    auto length = [](const Tile& t) { return THREADS - 1 - min(max(t.hi - t.lo, 0) / 128, THREADS - 1); };
    s_place[tid] = 0;
    __syncthreads();
    for (int i = tid; i < n_tiles; i += THREADS) atomicAdd(&s_place[length(tile(i))], 1);
    __syncthreads();
    const int count = s_place[tid];
    int before = count;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xFFFFFFFFu, before, o);
      if (lane >= o) before += v;
    }
    if (lane == 31) s_step_warp[w] = before;
    __syncthreads();
    before -= count;
    for (int v = 0; v < w; ++v) before += (int)s_step_warp[v];
    s_place[tid] = before;
    __syncthreads();
    for (int i = tid; i < n_tiles; i += THREADS) {
      const Tile t = tile(i);
      P.tiles[atomicAdd(&s_place[length(t)], 1)] = t;
    }
  }
  if (tid == 0) {
    P.header->status = s_bad;
    P.header->n_tiles = n_tiles;
    P.header->share = share;
  }
}

// ------------------------------------------------------------------------------ rows

// D[16 x 8] += A[16 x 16] B[16 x 8], fp16 operands, fp32 sums
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// transpose of an 8 x 8 matrix of 16-bit values held two to a lane
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}


// One warp's share of the steps of a unit (one request or tile, one KV head).
//
// The two products are taken with the cached tokens as the rows of the matrix instruction:
// S^T[16 tokens x 8 rows] = K Q^T and O^T[16 dims x 8 rows] += V^T P^T, so that 8 query
// rows fill an instruction (16 would be needed with the roles exchanged), and codes go
// from global memory to the operand's registers without shared memory: the contraction's
// order is free, so a lane's 16 consecutive key bytes are its operands of four
// instructions, and its 16 consecutive value bytes of four tokens are its operands of
// eight.  P^T comes from S^T's registers by an 8 x 8 transpose.
//
// Lane r * 4 + c (r = lane / 4, c = lane % 4) holds, for tile nt of 8 rows, the scores of
// tokens r and r + 8 for rows 8 nt + 2c and + 1; and O^T of dims r * (D / 8) + 0 .. D / 8 - 1
// for the same rows.
template <int D, int NT>
struct RowState {
  float o[NT][D / 16][4];
  float m[NT][2], l[NT][2];
};

template <int D>
struct Codes {
  uint4 k[2][D / 64];   // token r (0) and r + 8 (1): bytes 64 j + 16 c ..
  uint4 v[4];           // tokens 2c, 2c + 1, 2c + 8, 2c + 9: bytes r * (D / 8) .. (8 of them for D = 64)
};

// The steps of one warp: every `stride`-th one of [first, end).  A warp stops at the first
// use of a value that it is still loading, so a step's table entry is loaded three steps
// ahead and looked at one step later, when its codes are sent for to L2; codes and scales
// are loaded one step ahead.
template <int D>
struct Steps {
  const Params& P;
  const int32_t* table;
  int head, lo, hi, first, end, stride;
  const uint8_t *k_lane, *v_lane;   // the pools at the lane's place in a step
  Codes<D> C;
  int page, raw_next, raw_after;   // the first step's page, the entries of the two behind it
  float ks, vs;

  __device__ __forceinline__ int entry(int s) const {
    const int base = lo + s * STEP;
    return (s < end && base < hi) ? __ldg(table + (base >> P.page_shift)) : -1;
  }
  __device__ __forceinline__ int valid(int raw) const { return (raw < 0 || raw >= P.n_pages) ? -1 : raw; }
  // first row of a step in the pools
  __device__ __forceinline__ uint32_t row_of(int page_, int s) const {
    return (((uint32_t)page_ * P.h_kv + head) << P.page_shift) + ((lo + s * STEP) & ((1 << P.page_shift) - 1));
  }
  __device__ __forceinline__ void load_k(int page_, int s) {
    if (page_ < 0) return;
    const uint8_t* k = k_lane + (uint64_t)row_of(page_, s) * D;
#pragma unroll
    for (int j = 0; j < D / 64; ++j) {
      C.k[0][j] = dsa::ldg_nc(k + 64 * j);
      C.k[1][j] = dsa::ldg_nc(k + 8 * D + 64 * j);
    }
  }
  __device__ __forceinline__ void load_v(int page_, int s) {
    if (page_ < 0) return;
    const uint8_t* v = v_lane + (uint64_t)row_of(page_, s) * D;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint8_t* at = v + ((i & 1) + (i >> 1) * 8) * D;
      if (D == 128) {
        C.v[i] = dsa::ldg_nc(at);
      } else {
        const uint2 x = dsa::ldg_nc_v2(at);
        C.v[i] = make_uint4(x.x, x.y, 0u, 0u);
      }
    }
  }
  __device__ __forceinline__ float load_scale(const float* scale, int page_) const {
    return page_ < 0 ? 1.0f : __ldg(scale + (uint64_t)((uint32_t)page_ * P.h_kv + head));
  }
  // two parts, so that the queries can be fetched between them
  __device__ __forceinline__ void begin() {
    page = entry(first);
    raw_next = entry(first + stride);
    raw_after = entry(first + 2 * stride);
  }
  // a step's codes from memory to L2: a lane for each of their lines
  __device__ __forceinline__ void prefetch(int page_, int s) const {
    constexpr int LINES = STEP * D / 128;   // of the keys, and of the values
    const int lane = threadIdx.x & 31;
    if (page_ < 0 || lane >= 2 * LINES) return;
    const uint8_t* at = (lane < LINES ? P.k_pool : P.v_pool) + (uint64_t)row_of(page_, s) * D + (lane % LINES) * 128;
    dsa::prefetch_line_l2(at);
  }
  __device__ __forceinline__ void load_first() {
    page = valid(page);
    load_k(page, first);
    load_v(page, first);
    ks = load_scale(P.k_scale, page);
    vs = load_scale(P.v_scale, page);
  }
};

template <int D, int NT>
__device__ __forceinline__ void rows_steps(const Params& P, Steps<D>& W, int seen_lo,
                                           const uint32_t (&qf)[NT == 1 ? D / 16 : 1][2], const uint16_t* s_q,
                                           const float (&qs)[NT][2], const int (&pos)[NT][2], int pos_min, int pos_max,
                                           RowState<D, NT>& R) {
  const int lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
  const int lo = W.lo, hi = W.hi, stride = W.stride;
  Codes<D>& C = W.C;
  int page = W.page, raw_next = W.raw_next, raw_after = W.raw_after;
  float ks = W.ks, vs = W.vs;
  // The registers have room for one step ahead, L2 for two.  us, with and without: 64
  // requests of up to 32k tokens 309 and 317, 48 of up to 8k with 4 queries 89 and 93, 32
  // rows 101 and 107; but one row tile in a wide CTA, which has few steps, 19.8 and 19.4.
  const bool prefetch = NT > 1 || stride == ROW_WARPS;
  for (int s = W.first; s < W.end; s += stride) {
    const int page_next = W.valid(raw_next);
    raw_next = raw_after;
    raw_after = W.entry(s + 3 * stride);
    if (prefetch) W.prefetch(W.valid(raw_next), s + 2 * stride);
    const float ks_next = W.load_scale(P.k_scale, page_next), vs_next = W.load_scale(P.v_scale, page_next);
    if (page < 0) {
      W.load_k(page_next, s + stride);
      W.load_v(page_next, s + stride);
    } else {
      const int base = lo + s * STEP;
      // scores
      float x[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) x[nt][e] = 0.f;
#pragma unroll
      for (int j = 0; j < D / 64; ++j) {
        uint32_t qw[NT][8];
        if (NT > 1) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const uint4* at = reinterpret_cast<const uint4*>(s_q + (8 * nt + r) * (D + 8) + 64 * j + 16 * c);
            const uint4 a = at[0], b = at[1];
            qw[nt][0] = a.x; qw[nt][1] = a.y; qw[nt][2] = a.z; qw[nt][3] = a.w;
            qw[nt][4] = b.x; qw[nt][5] = b.y; qw[nt][6] = b.z; qw[nt][7] = b.w;
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t w0 = word(C.k[0][j], i), w1 = word(C.k[1][j], i);
          const uint32_t a0 = dsa::e4m3x2_to_f16x2(w0 & 0xFFFFu), a2 = dsa::e4m3x2_to_f16x2(w0 >> 16);
          const uint32_t a1 = dsa::e4m3x2_to_f16x2(w1 & 0xFFFFu), a3 = dsa::e4m3x2_to_f16x2(w1 >> 16);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            if (NT == 1) mma(x[nt], a0, a1, a2, a3, qf[4 * j + i][0], qf[4 * j + i][1]);
            else mma(x[nt], a0, a1, a2, a3, qw[nt][2 * i], qw[nt][2 * i + 1]);
          }
        }
      }
      W.load_k(page_next, s + stride);
      // t = x + log2(v_scale), masked
      const float vsc = bounded_scale(vs);
      float bias, vinv;   // 2^-22 relative, as the exponential
      asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(bias) : "f"(vsc));
      asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(vinv) : "f"(vsc));
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) x[nt][e] = fmaf(x[nt][e], qs[nt][e & 1] * ks, bias);
      const bool edge = base + STEP - 1 > pos_min || (P.window > 0 && base <= pos_max - P.window);
      if (edge) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int j = base + r + (e >> 1) * 8, p = pos[nt][e & 1];
            if (j > p || (P.window > 0 && j <= p - P.window)) x[nt][e] = -INFINITY;
          }
        // rows outside what any query sees may hold NaN codes: 0 * NaN is not 0
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int j = base + 2 * c + (i & 1) + (i >> 1) * 8;
          if (j < seen_lo || j >= hi) C.v[i] = make_uint4(0u, 0u, 0u, 0u);
        }
      }
      // the running maximum, moved only when a score passes it by 2^LAG, and for every page of a small
      // value scale, whose part of the sum is formed there
      bool up = vsc < SMALL_SCALE;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) up |= fmaxf(x[nt][e], x[nt][e + 2]) > R.m[nt][e] + LAG;
      if (__any_sync(0xFFFFFFFFu, up)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float f[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float t = fmaxf(fmaxf(x[nt][e], x[nt][e + 2]), R.m[nt][e]);
#pragma unroll
            for (int o = 4; o <= 16; o <<= 1) t = fmaxf(t, __shfl_xor_sync(0xFFFFFFFFu, t, o));
            f[e] = ex2(R.m[nt][e] - t);
            R.l[nt][e] = scaled(R.l[nt][e], R.m[nt][e] - t);
            R.m[nt][e] = t;
          }
#pragma unroll
          for (int mt = 0; mt < D / 16; ++mt)
#pragma unroll
            for (int e = 0; e < 4; ++e) R.o[nt][mt][e] *= f[e & 1];
        }
        if (vsc < SMALL_SCALE) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) R.l[nt][e & 1] += ex2(x[nt][e] - R.m[nt][e & 1] - bias);
          vinv = 0.f;
        }
      }
      uint32_t pf[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float wt[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) wt[e] = ex2(x[nt][e] - R.m[nt][e & 1]);
        R.l[nt][0] = fmaf(wt[0] + wt[2], vinv, R.l[nt][0]);
        R.l[nt][1] = fmaf(wt[1] + wt[3], vinv, R.l[nt][1]);
        pf[nt][0] = transpose8(dsa::pack_f16x2(wt[0], wt[1]));
        pf[nt][1] = transpose8(dsa::pack_f16x2(wt[2], wt[3]));
      }
      // values
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const uint32_t w0 = word(C.v[0], i), w1 = word(C.v[1], i), w2 = word(C.v[2], i), w3 = word(C.v[3], i);
        const uint32_t p0 = __byte_perm(w0, w1, 0x5140), p1 = __byte_perm(w0, w1, 0x7362);
        const uint32_t p2 = __byte_perm(w2, w3, 0x5140), p3 = __byte_perm(w2, w3, 0x7362);
        const uint32_t a[2][4] = {
            {dsa::e4m3x2_to_f16x2(p0 & 0xFFFFu), dsa::e4m3x2_to_f16x2(p0 >> 16), dsa::e4m3x2_to_f16x2(p2 & 0xFFFFu),
             dsa::e4m3x2_to_f16x2(p2 >> 16)},
            {dsa::e4m3x2_to_f16x2(p1 & 0xFFFFu), dsa::e4m3x2_to_f16x2(p1 >> 16), dsa::e4m3x2_to_f16x2(p3 & 0xFFFFu),
             dsa::e4m3x2_to_f16x2(p3 >> 16)}};
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            mma(R.o[nt][2 * i + h], a[h][0], a[h][1], a[h][2], a[h][3], pf[nt][0], pf[nt][1]);
      }
      W.load_v(page_next, s + stride);
    }
    page = page_next;
    ks = ks_next;
    vs = vs_next;
  }
}

template <int D, int NT, int NW>
struct RowSmem {
  static constexpr int PITCH = D + 4;   // floats of a row: the warps' writes meet no bank conflict
  float o[NW][8 * NT][PITCH];
  float m[NW][8 * NT], l[NW][8 * NT];
  uint16_t q[NT == 1 ? 8 : 8 * NT * (D + 8)];
  float q_scale[8 * NT];
  int last;
  Share share;
  long long scan[NW], share_steps;
};

__device__ __forceinline__ void wait_for_plan() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Steps [step0, step1) of one unit by the whole CTA, joined over its warps.  Rows
// [row0, row0 + 8 NT) of the request.  The unit is in `pieces`, which CTAs first_cta,
// first_cta + 1, ... have; this CTA has piece `piece`.  A unit in one piece goes to `out`.
// Else the pieces go to partial buffers, and the last CTA to arrive in each group of JOIN
// pieces joins the group, and the last of those the groups: always in the order of the
// pieces, so that the result does not depend on which one it was.
//
// A CTA has four partial buffers: for the piece of a unit that it began (1) or continued
// (0), and for the group of pieces that it is the first of (3, 2).
template <int D, int NT, int NW>
__device__ __forceinline__ void rows_unit(const Params& P, RowSmem<D, NT, NW>& S, int req, const Request& a, int head,
                                          int row0, const Span& sp, int step0, int step1, int pieces, int first_cta,
                                          int piece) {
  constexpr int R8 = 8 * NT;
  constexpr int PSIZE = R8 * D + 2 * R8;   // floats of one partial result
  constexpr int JOIN = NW > ROW_WARPS ? 32 : 16;   // partial results that one CTA joins at a time
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5, r = lane >> 2, c = lane & 3;
  const int rows = a.rows(P);
  const int pos0 = a.kv - a.q_len;

  const int pos_min = pos0 + row0 / P.group, pos_max = pos0 + min(row0 + R8 - 1, rows - 1) / P.group;
  const int hi = min(pos_max + 1, a.kv);
  const int seen_lo = P.window > 0 ? max(pos_min - P.window + 1, 0) : 0;
  Steps<D> W{P, P.table + req * P.table_ld, head, sp.lo, hi, step0 + w, step1, NW,
             P.k_pool + r * D + 16 * c, P.v_pool + 2 * c * D + r * (D / 8)};
  W.begin();

  // queries: fp16 after a scaling of each row by a power of two that brings its largest
  // magnitude to [2^7, 2^8).  Every warp keeps a single tile of rows in registers; of
  // several, a warp prepares one for all.
  uint32_t qf[NT == 1 ? D / 16 : 1][2];
  float qs[NT][2];
  int pos[NT][2];
  float scale_row = 1.0f;
  static_assert(NW >= NT, "a warp for each tile of rows");
  if (NT == 1 || w < NT) {
    const int nt = NT == 1 ? 0 : w;
    const int row = row0 + 8 * nt + r;
    uint4 v[D / 64][2];
    float mx = 0.f;
    const bool in = row < rows;
    const int i = row / P.group;
    const uint16_t* src = P.q + (a.q0 + i) * P.q_ld + (head * P.group + row - i * P.group) * P.q_hd + 16 * c;
#pragma unroll
    for (int j = 0; j < D / 64; ++j)
#pragma unroll
      for (int h = 0; h < 2; ++h) v[j][h] = in ? dsa::ldg_nc(src + 64 * j + 8 * h) : make_uint4(0u, 0u, 0u, 0u);
    W.load_first();
#pragma unroll
    for (int j = 0; j < D / 64; ++j)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 f = unpack(word(v[j][h], e), P.fp16);
          mx = fmaxf(mx, fmaxf(fabsf(f.x), fabsf(f.y)));
        }
    mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 1));
    mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 2));
    const float down = row_scaling(mx, scale_row);
#pragma unroll
    for (int j = 0; j < D / 64; ++j)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t p[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const float2 f = unpack(word(v[j][h], u), P.fp16);
          p[u] = dsa::pack_f16x2(f.x * down, f.y * down);
        }
        if (NT == 1) {
          qf[NT == 1 ? 4 * j + 2 * h : 0][0] = p[0];
          qf[NT == 1 ? 4 * j + 2 * h : 0][1] = p[1];
          qf[NT == 1 ? 4 * j + 2 * h + 1 : 0][0] = p[2];
          qf[NT == 1 ? 4 * j + 2 * h + 1 : 0][1] = p[3];
        } else {
          *reinterpret_cast<uint4*>(S.q + (8 * nt + r) * (D + 8) + 64 * j + 16 * c + 8 * h) = make_uint4(p[0], p[1], p[2], p[3]);
        }
      }
    if (NT > 1 && c == 0) S.q_scale[8 * nt + r] = scale_row;
  } else {
    W.load_first();
  }
  if (NT > 1) __syncthreads();
  // this lane's score columns are rows 8 nt + 2c + e
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float back = NT == 1 ? __shfl_sync(0xFFFFFFFFu, scale_row, (2 * c + e) * 4) : S.q_scale[8 * nt + 2 * c + e];
      qs[nt][e] = back * P.scale_log2;
      pos[nt][e] = pos0 + min(row0 + 8 * nt + 2 * c + e, rows - 1) / P.group;
    }

  RowState<D, NT> R;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int mt = 0; mt < D / 16; ++mt)
#pragma unroll
      for (int e = 0; e < 4; ++e) R.o[nt][mt][e] = 0.f;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      R.m[nt][e] = M_INIT;
      R.l[nt][e] = 0.f;
    }
  }
  rows_steps<D, NT>(P, W, seen_lo, qf, S.q, qs, pos, pos_min, pos_max, R);

  // join the warps: dims are kept in the order mt * 16 + r * 2 + (0, 1)
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float l = R.l[nt][e];
#pragma unroll
      for (int o = 4; o <= 16; o <<= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, o);
      const int row = 8 * nt + 2 * c + e;
      if (r == 0) {
        S.m[w][row] = R.m[nt][e];
        S.l[w][row] = l;
      }
#pragma unroll
      for (int mt = 0; mt < D / 16; ++mt)
        *reinterpret_cast<float2*>(&S.o[w][row][mt * 16 + r * 2]) = make_float2(R.o[nt][mt][e], R.o[nt][mt][e + 2]);
    }
  __syncthreads();
  const int live = min(rows - row0, R8);
  auto buffer = [&](int p, int group) -> float* {
    return P.partial + (4LL * (first_cta + p) + 2 * group + (p == 0 ? 1 : 0)) * PSIZE;
  };
  float* mine = pieces > 1 ? buffer(piece, 0) : nullptr;
  auto write = [&](int row, int k4, float4 o, float m, float l) {
    // o: dims k4 .. k4 + 3 in the joined order, which are two pairs of neighbours
    const int i = (row0 + row) / P.group, h = head * P.group + (row0 + row) - i * P.group;
    const float inv = l > 0.f ? 1.0f / l : (l == 0.f ? 0.f : l);   // a NaN sum stays one
    const int mt = k4 >> 4, rr = (k4 & 15) >> 1;
    uint16_t* at = P.out + (a.q0 + i) * P.out_ld + h * P.out_hd + rr * (D / 8) + 2 * mt;
    *reinterpret_cast<uint32_t*>(at) = pack(o.x * inv, o.y * inv, P.fp16);
    *reinterpret_cast<uint32_t*>(at + D / 8) = pack(o.z * inv, o.w * inv, P.fp16);
    if (k4 == 0 && P.lse)
      P.lse[(long long)(a.q0 + i) * P.h_q + h] = l == 0.f ? -INFINITY : 0.6931471805599453f * (m + log2f(l));
  };
  for (int u = tid; u < live * (D / 4); u += 32 * NW) {
    const int row = u / (D / 4), k4 = (u % (D / 4)) * 4;
    float m = S.m[0][row];
#pragma unroll
    for (int x = 1; x < NW; ++x) m = fmaxf(m, S.m[x][row]);
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    float l = 0.f;
#pragma unroll
    for (int x = 0; x < NW; ++x) {
      const float f = ex2(S.m[x][row] - m);
      const float4 v = *reinterpret_cast<const float4*>(&S.o[x][row][k4]);
      o.x = fmaf(v.x, f, o.x);
      o.y = fmaf(v.y, f, o.y);
      o.z = fmaf(v.z, f, o.z);
      o.w = fmaf(v.w, f, o.w);
      l += scaled(S.l[x][row], S.m[x][row] - m);
    }
    if (pieces == 1) {
      write(row, k4, o, m, l);
    } else {
      *reinterpret_cast<float4*>(mine + row * D + k4) = o;
      if (k4 == 0) {
        mine[R8 * D + row] = m;
        mine[R8 * D + R8 + row] = l;
      }
    }
  }
  if (pieces > 1) {
    // join pieces p0, p0 + by, ... (n of them, of this kind of buffer) into `to`, or into the result
    auto join = [&](int p0, int by, int n, int group, float* to) {
      for (int u = tid; u < live * (D / 4); u += 32 * NW) {
        const int row = u / (D / 4), k4 = (u % (D / 4)) * 4;
        float m = M_INIT, l = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int x0 = 0; x0 < n; x0 += 8) {
          float pm[8], pl[8];
          float4 po[8];
#pragma unroll
          for (int x = 0; x < 8; ++x) {
            pm[x] = M_INIT;
            pl[x] = 0.f;
            po[x] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (x0 + x < n) {
              const float* b = buffer(p0 + (x0 + x) * by, group);
              po[x] = __ldcg(reinterpret_cast<const float4*>(b + row * D + k4));
              pm[x] = __ldcg(b + R8 * D + row);
              pl[x] = __ldcg(b + R8 * D + R8 + row);
            }
          }
          float top = m;
#pragma unroll
          for (int x = 0; x < 8; ++x) top = fmaxf(top, pm[x]);
          const float f0 = ex2(m - top);
          o.x *= f0; o.y *= f0; o.z *= f0; o.w *= f0;
          l = scaled(l, m - top);
#pragma unroll
          for (int x = 0; x < 8; ++x) {
            const float f = ex2(pm[x] - top);
            o.x = fmaf(po[x].x, f, o.x);
            o.y = fmaf(po[x].y, f, o.y);
            o.z = fmaf(po[x].z, f, o.z);
            o.w = fmaf(po[x].w, f, o.w);
            l += scaled(pl[x], pm[x] - top);
          }
          m = top;
        }
        if (!to) {
          write(row, k4, o, m, l);
        } else {
          *reinterpret_cast<float4*>(to + row * D + k4) = o;
          if (k4 == 0) {
            to[R8 * D + row] = m;
            to[R8 * D + R8 + row] = l;
          }
        }
      }
    };
    // whether this CTA is the last of n to come to a counter
    auto arrive = [&](int* counter, int n) -> bool {
      __threadfence();
      __syncthreads();
      if (tid == 0) S.last = atomicAdd(counter, 1) == n - 1;
      __syncthreads();
      const bool last = S.last != 0;
      if (last) __threadfence();
      return last;
    };
    wait_for_plan();   // it sets the counters
    const int groups = (pieces + JOIN - 1) / JOIN, lead = piece / JOIN * JOIN;
    if (arrive(P.arrived + 3 * (first_cta + lead) + (lead == 0 ? 1 : 0), min(JOIN, pieces - lead))) {
      join(lead, 1, min(JOIN, pieces - lead), 0, groups > 1 ? buffer(lead, 1) : nullptr);
      if (groups > 1 && arrive(P.arrived + 3 * first_cta + 2, groups)) join(0, JOIN, groups, 1, nullptr);
    }
  }
  __syncthreads();   // the shared memory is used again
}

// This CTA's share, and in share_steps the steps of each share: what the plan kernel
// computes.  A thread looks at P.own_plan requests.
template <int D, int NT, int NW>
__device__ __forceinline__ Share own_share(const Params& P, RowSmem<D, NT, NW>& S, int b) {
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int r0 = min(tid * P.own_plan, P.n_req), r1 = min(r0 + P.own_plan, P.n_req);
  long long steps = 0;
  for (int r = r0; r < r1; ++r) steps += unit_steps(P, request(P, r));
  if (tid == 0) S.share = Share{-1, 0, 0};
  long long in = steps;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long v = __shfl_up_sync(0xFFFFFFFFu, in, o);
    if (lane >= o) in += v;
  }
  if (lane == 31) S.scan[w] = in;
  __syncthreads();
  long long before = in - steps, all = 0;
#pragma unroll
  for (int u = 0; u < NW; ++u) {
    if (u < w) before += S.scan[u];
    all += S.scan[u];
  }
  const long long share = share_of(P, all * P.h_kv), f = b * share;
  if (before * P.h_kv <= f && f < (before + steps) * P.h_kv)
    for (int r = r0; r < r1; ++r) {
      const long long here = unit_steps(P, request(P, r));
      if (f < (before + here) * P.h_kv) {
        S.share = share_at(P, r, f - before * P.h_kv, here);
        break;
      }
      before += here;
    }
  if (tid == 0) S.share_steps = share;
  __syncthreads();
  return S.share;
}

template <int D, int NT, int NW>
__device__ __forceinline__ void rows_share(const Params& P, RowSmem<D, NT, NW>& S) {
  const int b = blockIdx.x;
  Share at;
  long long share;
  if (P.own_plan) {
    at = own_share(P, S, b);
    share = S.share_steps;
  } else {
    wait_for_plan();
    at = P.shares[b];
    share = P.header->share;
  }
  int req = at.req, head = at.head;
  if (req < 0) return;
  long long step = at.step, left = share;   // step: of the unit, below 0 in its beginning
  long long unit = b * share - step;        // where the unit's steps begin among all
  Request a = request(P, req);
  Span sp = span(P, a, 0, a.q_len - 1);
  while (true) {
    // the next request's lengths, while this unit is computed
    int next[3] = {0, 0, 0};
    if (head + 1 == P.h_kv && req + 1 < P.n_req) {
      next[0] = __ldg(P.cu_q + req + 1);
      next[1] = __ldg(P.cu_q + req + 2);
      next[2] = __ldg(P.kv_lens + req + 1);
    }
    const int s0 = (int)max(step, 0LL), s1 = (int)min((long long)sp.steps, step + left);
    if (s0 < s1) {
      const int first = (int)(unit / share), last = (int)((unit + sp.steps - 1) / share);
      rows_unit<D, NT, NW>(P, S, req, a, head, 0, sp, s0, s1, last - first + 1, first, b - first);
    }
    left -= min(left, sp.steps - step);
    if (left == 0) return;
    unit += sp.steps + P.unit_steps;
    step = -P.unit_steps;
    if (++head < P.h_kv) continue;
    head = 0;
    if (++req >= P.n_req) return;
    a = request(P, next[0], next[1], next[2]);
    while (a.q_len == 0 || a.q_len > P.max_q_len || a.rows(P) > P.small_rows) {
      if (++req >= P.n_req) return;
      a = request(P, req);
    }
    sp = span(P, a, 0, a.q_len - 1);
  }
}

template <int D, int NT, int NW>
__global__ void __launch_bounds__(32 * NW, NW > ROW_WARPS ? 1 : ctas_per_sm(D, NT)) rows_kernel(const __grid_constant__ Params P) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // the tiles' kernel, if there is one
  rows_share<D, NT, NW>(P, *reinterpret_cast<RowSmem<D, NT, NW>*>(smem_raw));
  wait_for_plan();   // what waits for this kernel needs the plan
}

// ------------------------------------------------------------------------------ host
static bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

static int check(const dsa_kv8_params* p) {
  if (!p || p->n_tokens < 0 || p->n_tokens > (1 << 30) || p->n_req < 0 || p->h_q < 1 || p->h_kv < 1 ||
      p->h_q % p->h_kv != 0 || p->n_pages < 0 || p->table_cols < 0 || p->max_q_len < 0 || p->window < 0 ||
      (p->type != DSA_KV8_BF16 && p->type != DSA_KV8_FP16) || !isfinite(p->softmax_scale) ||
      (p->flags & ~DSA_KV8_FLAG_TEST_WAIT_TIMEOUT) != 0)
    return DSA_ERR_INVALID_ARG;
  if ((p->d != 64 && p->d != 128) ||
      (p->page_size != 16 && p->page_size != 32 && p->page_size != 64 && p->page_size != 128) ||
      p->n_req > DSA_KV8_MAX_REQ || p->h_kv > DSA_KV8_MAX_HEADS || p->h_q / p->h_kv > DSA_KV8_MAX_GROUP ||
      (long long)p->n_tokens * (p->h_q / p->h_kv) >= (1LL << 31) ||
      (long long)p->n_pages * p->h_kv * p->page_size >= (1LL << 32) - 1 ||   // rows of a pool are numbered in 32 bits
      (p->window > (1 << 30) && (long long)p->table_cols * p->page_size > (1LL << 30)))
    return DSA_ERR_UNSUPPORTED_SHAPE;
  return DSA_OK;
}

// tiles of 8 query rows of a request in rows_kernel: 1, 2 or 4.  Where the batch has
// requests for the tiles as well, single-query requests set it.
static int row_tiles(const dsa_kv8_params* p) {
  const long long group = p->h_q / p->h_kv, most = (long long)p->max_q_len * group;
  const long long rows = most <= MAX_ROWS ? most : (group <= MAX_ROWS ? group : MAX_ROWS);
  return rows <= 8 ? 1 : rows <= 16 ? 2 : 4;
}

// whether a request may have more rows than rows_kernel takes
static bool has_tiles(const dsa_kv8_params* p) {
  return (long long)p->max_q_len * (p->h_q / p->h_kv) > 8 * row_tiles(p);
}

// Whether a CTA of rows_kernel has all the warps that an SM holds, or four of them.  The lengths are
// on the GPU, so the rule goes by the most that a request may have, the table's columns; the figures
// are for tables as wide as the longest request, and a wider one takes the wide CTAs' figure.  With
// few units, which many CTAs share, wider CTAs leave fewer pieces to join; with short ones
// their warps have nothing to do.  Heads of 128, 64/8 heads, us, wide and not: 4 requests of
// up to 2500 tokens 14.6 and 13.2, 4000 15.2 and 17.3, 12000 17.9 and 21.9; 8 of 2500 15.1
// and 13.7, 4000 15.2 and 17.7; 16 (128 units) of 2k 16.0 and 14.3.  Heads of 64 (24 warps):
// 12 of up to 4k tokens, 16/4 heads, 14.2 and 11.5.
static bool wide(const dsa_kv8_params* p, int sms) {
  const long long units = (long long)p->n_req * p->h_kv;
  long long most = (long long)p->table_cols * p->page_size;   // cached tokens that a request's queries see
  if (p->window > 0 && most > (long long)p->window + p->max_q_len) most = (long long)p->window + p->max_q_len;
  return p->d == 128 && 2 * units <= sms && most >= 3500;
}

struct Layout {
  int n_shares, max_tiles;
  size_t shares, arrived, tiles, partial, bytes;
};

static size_t up(size_t x) { return (x + 255) / 256 * 256; }

static Layout layout(const dsa_kv8_params* p, int sms) {
  Layout L;
  const size_t group = p->h_q / p->h_kv, rows = 8 * (size_t)row_tiles(p);
  L.n_shares = wide(p, sms) ? sms : ctas_per_sm(p->d, row_tiles(p)) * sms;
  size_t at = 256;
  L.shares = at;
  at += up(L.n_shares * sizeof(Share));
  L.arrived = at;
  at += up(L.n_shares * 3 * sizeof(int));
  L.tiles = at;
  L.max_tiles = (int)((p->n_tokens * group + (TILE_ROWS - 1) * (size_t)p->n_req) / TILE_ROWS);   // ascending cu_q cannot give more
  at += up((size_t)L.max_tiles * sizeof(Tile));
  L.partial = at;
  at += up((size_t)L.n_shares * 4 * (rows * p->d + 2 * rows) * sizeof(float));
  L.bytes = at;
  return L;
}

// `most` is the most dynamic shared memory that any call asks of the kernel.  The limit is set to
// that and never to less: another host thread may set it between this one's setting and its launch.
template <typename K>
static int launch(K kernel, int grid, int threads, size_t smem, size_t most, cudaStream_t st, const Params& P, bool dependent) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = dependent ? 1 : 0;
  // the limit of 48 KB is for dynamic and static shared memory together; no kernel here has 8 KB of the latter
  if (smem > 40 * 1024 && cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most) != cudaSuccess)
    return DSA_ERR_CUDA;
  return cudaLaunchKernelEx(&cfg, kernel, P) == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}

template <int D, int NT>
static int launch_rows(const Params& P, bool wide, cudaStream_t st) {
  constexpr int W = ROW_WARPS, WW = D == 128 ? W * ctas_per_sm(D, NT) : W;
  constexpr size_t smem = sizeof(RowSmem<D, NT, W>), wide_smem = sizeof(RowSmem<D, NT, WW>);
  return wide ? launch(rows_kernel<D, NT, WW>, P.n_shares, 32 * WW, wide_smem, wide_smem, st, P, true)
              : launch(rows_kernel<D, NT, W>, P.n_shares, 32 * W, smem, smem, st, P, true);
}

template <int D>
static int launch_all(const dsa_kv8_params* p, const Params& P, bool wide, cudaStream_t st) {
  const int nt = row_tiles(p);
  const int rc = nt == 1 ? launch_rows<D, 1>(P, wide, st) : nt == 2 ? launch_rows<D, 2>(P, wide, st) : launch_rows<D, 4>(P, wide, st);
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

static int current_sms(int* sms) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return DSA_ERR_CUDA;
  return cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}

size_t dsa_kv8_attn_workspace_size(const dsa_kv8_params* p, int num_sms) {
  if (dsa_kv8::check(p) != DSA_OK) return 0;
  if (num_sms <= 0 && current_sms(&num_sms) != DSA_OK) return 0;
  return dsa_kv8::layout(p, num_sms).bytes;
}

int dsa_kv8_attn_fwd(const void* q, int64_t q_ld, int64_t q_hd, const void* k_pool, const void* v_pool,
                     const float* k_scale, const float* v_scale, const int32_t* block_table, int64_t table_ld,
                     const int32_t* cu_q, const int32_t* kv_lens, void* out, int64_t out_ld, int64_t out_hd, float* lse,
                     const dsa_kv8_params* p, void* workspace, size_t workspace_bytes, void* stream) {
  using namespace dsa_kv8;
  const int rc = check(p);
  if (rc != DSA_OK) return rc;
  if (!workspace || !aligned(workspace, 256)) return DSA_ERR_INVALID_ARG;
  if (p->n_tokens > 0 && p->n_req > 0) {
    if (q_ld % 8 != 0 || q_hd % 8 != 0 || out_ld % 8 != 0 || out_hd % 8 != 0 || q_ld < p->d || out_ld < p->d ||
        (p->h_q > 1 && (q_hd < p->d || out_hd < p->d)) || table_ld < p->table_cols)
      return DSA_ERR_INVALID_ARG;
    if (!q || !out || !cu_q || !kv_lens || !aligned(q, 16) || !aligned(out, 16) || !aligned(cu_q, 4) ||
        !aligned(kv_lens, 4) || !aligned(lse, 4))
      return DSA_ERR_INVALID_ARG;
    if (p->table_cols > 0 && (!block_table || !aligned(block_table, 4))) return DSA_ERR_INVALID_ARG;
    if (p->n_pages > 0 && (!k_pool || !v_pool || !k_scale || !v_scale || !aligned(k_pool, 16) || !aligned(v_pool, 16) ||
                           !aligned(k_scale, 4) || !aligned(v_scale, 4)))
      return DSA_ERR_INVALID_ARG;
  }
  int dev = 0, major = 0, minor = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return DSA_ERR_CUDA;
  cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev);
  cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev);
  if (major != 10 || minor != 3) return DSA_ERR_UNSUPPORTED_DEVICE;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return DSA_ERR_CUDA;
  const Layout L = layout(p, sms);
  if (workspace_bytes < L.bytes) return DSA_ERR_WORKSPACE_TOO_SMALL;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  cudaStream_t st = (cudaStream_t)stream;
  if (p->n_tokens == 0 || p->n_req == 0)
    return cudaMemsetAsync(ws, 0, sizeof(uint32_t), st) == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
  Params P;
  P.q = static_cast<const uint16_t*>(q);
  P.k_pool = static_cast<const uint8_t*>(k_pool);
  P.v_pool = static_cast<const uint8_t*>(v_pool);
  P.k_scale = k_scale;
  P.v_scale = v_scale;
  P.table = block_table;
  P.cu_q = cu_q;
  P.kv_lens = kv_lens;
  P.out = static_cast<uint16_t*>(out);
  P.lse = lse;
  P.q_ld = q_ld;
  P.q_hd = q_hd;
  P.out_ld = out_ld;
  P.out_hd = out_hd;
  P.table_ld = table_ld;
  P.header = reinterpret_cast<Header*>(ws);
  P.shares = reinterpret_cast<Share*>(ws + L.shares);
  P.arrived = reinterpret_cast<int*>(ws + L.arrived);
  P.tiles = reinterpret_cast<Tile*>(ws + L.tiles);
  P.partial = reinterpret_cast<float*>(ws + L.partial);
  P.n_tokens = p->n_tokens;
  P.n_req = p->n_req;
  P.h_q = p->h_q;
  P.h_kv = p->h_kv;
  P.group = p->h_q / p->h_kv;
  P.n_pages = p->n_pages;
  P.page_shift = __builtin_ctz(p->page_size);
  // positions stay below 2^31 with room for a step and a tile behind the last one
  const long long cap = (long long)p->table_cols * p->page_size, most = (1LL << 31) - 1024;
  P.cap = (int)(cap < most ? cap : most);
  P.max_q_len = p->max_q_len;
  // a window that nothing passes is none; others stay where a position minus the window
  // (at least -2^30 minus 2^30) is an int
  P.window = p->window < P.cap ? p->window : 0;
  P.fp16 = p->type == DSA_KV8_FP16;
  P.has_tiles = has_tiles(p);
  // cached tokens that a tile's rows may see
  const long long seen = P.window > 0 ? (long long)P.window + TILE_ROWS / P.group + 1 + STEP : P.cap;
  const long long pairs = (long long)L.max_tiles * p->h_kv;
  P.cluster = P.has_tiles && 2 * pairs <= sms ? cluster_size(p->d, pairs, (int)((min(seen, (long long)P.cap) + 127) / 128)) : 0;
  P.n_ctas = P.cluster ? (int)pairs * P.cluster : sms;
  P.small_rows = 8 * row_tiles(p);
  P.n_shares = L.n_shares;
  const bool is_wide = wide(p, sms);
  const int warps = is_wide ? ROW_WARPS * ctas_per_sm(p->d, row_tiles(p)) : ROW_WARPS;
  P.unit_steps = UNIT_STEPS * warps;
  P.min_share = P.unit_steps + MIN_STEPS * warps;
  // the requests of a thread where the CTAs find their shares for themselves; 0: the plan kernel does
  P.own_plan = p->n_req <= OWN_PLAN * 32 * warps ? (p->n_req + 32 * warps - 1) / (32 * warps) : 0;
  P.max_tiles = L.max_tiles;
  P.test_block = p->flags & DSA_KV8_FLAG_TEST_WAIT_TIMEOUT ? 3u : 0xFFFFFFFFu;
  P.scale_log2 = p->softmax_scale * 1.4426950408889634f;
  const auto plan_smem = [](int n_req) { return (size_t)(n_req + 1) * 2 * sizeof(long long); };
  const size_t smem = plan_smem(p->n_req), most_smem = plan_smem(DSA_KV8_MAX_REQ);
  const int rc1 = P.own_plan ? launch(plan_kernel<FEW_THREADS>, 1, FEW_THREADS, smem, most_smem, st, P, false)
                             : launch(plan_kernel<PLAN_THREADS>, 1, PLAN_THREADS, smem, most_smem, st, P, false);
  if (rc1 != DSA_OK) return rc1;
  return p->d == 128 ? launch_all<128>(p, P, is_wide, st) : launch_all<64>(p, P, is_wide, st);
}

}  // extern "C"
