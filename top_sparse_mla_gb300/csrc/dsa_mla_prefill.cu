// Latent attention in its expanded form (include/dsa_mla_prefill.h): tiles of 256 query rows
// of a request and head, in two halves of 128, on the tensor cores (tcgen05).
//
// One persistent CTA per SM takes units (tile, head).  Roles:
//   - warps 0-3 and 4-7, a softmax group for each half: a thread owns a query row.  For each
//     block of 128 keys it reads its scores from tensor memory, forms the weights and writes
//     them back over the scores in the inputs' type; in the end it divides its row of O by the
//     softmax's sum and stores it;
//   - warp 8 copies queries, keys and values into shared memory (TMA, panels of 64 dims x 128
//     rows in the 128-byte swizzle): four panels for keys, which pass through three at a time
//     (128 dims of the head, 64 rotary ones), and two blocks of values;
//   - a thread of warp 9 issues the products: S = Q K^T (128 x 128 x 192) and O += P V (128 x 128 x
//     128, P in tensor memory).  The two halves alternate, so that one half's softmax runs under
//     the other half's products;
//   - warp 10 clears what a request's last block of values has behind the request's end.
// A tile with at most 128 rows is a unit of one half, and the halves take such units in turn: one's scores
// are formed while the other's values are.  Where several CTAs share one, both halves have its rows, and take
// the piece's blocks in turn.
//
// Work.  A one-CTA plan kernel lists the tiles.  With many units the longest come first and the CTAs take
// them forwards and backwards in turn.  With few (SPLIT), all units' blocks are laid in a row and cut into
// equal shares, one for each CTA: a unit that several CTAs share leaves partial results, which a last
// kernel joins.  A 2123-token prefill of 64 heads, 3.8 units an SM, took 185 us in shares and 118 in whole
// units.
//
// What bounds it.  6 chunks of up to 2048 queries on up to 8k keys, 32 heads: 763 us in a burst, 810 to 840 in
// a row (1320 TFLOP/s, 0.77 of a large bf16 product's sustained rate), at 1.35 kW, which holds the clock at
// 1.66 GHz.  A block of both halves takes 3400 cycles, its products 2560.  What is missing are the keys of the
// next block: beside 96 KB of queries shared memory holds 1.6 blocks, so that a copy has 1300 cycles of
// products to arrive in, and takes 2000.  (Sent for to L2 two to five blocks ahead they come no sooner, and
// five panels of keys beside one and a half blocks of values, 1500 cycles, change nothing: 849 us, and 72
// against 66 below.)  64 queries on 32k keys, 16 heads: 64 us, memory's part 40; the rest is the beginning, and
// the join of 10 pieces a unit.
//
// Every wait is bounded: where one runs out the call's status gets DSA_STATUS_WAIT_TIMEOUT
// and the CTA's roles stop, drain the tensor core and free its memory.
//
// Scores become u = S * (softmax_scale * log2 e) - m and weights 2^u, with m the maximum of the row's first
// scores, so that a row with one key has a weight of 1, which nothing rounds, and its value as it is.  m is
// raised, by whole numbers, and O rescaled by a power of two, exactly, when a weight would pass 2^15, so
// that each fits fp16: rare behind the first block.

#include <cuda.h>
#include <cuda_runtime.h>
#include <float.h>
#include <math.h>
#include <stdint.h>

#include <atomic>

#include "device.cuh"
#include "dsa_mla_prefill.h"
#include "ptx_sm103.cuh"

namespace dsa_mla {

using namespace dsa;

constexpr int DQ = 192, DN = 128, DR = 64, DV = 128;   // dims: a query's, its parts against k_nope and k_rope, a value's
constexpr int BLOCK = 128;         // keys of a block
constexpr int TILE_ROWS = 256;
constexpr int PANEL = 128 * 128;   // bytes of 64 dims of 128 rows
constexpr int K_PANELS = 4, V_BUFS = 2;
constexpr float MOST = 15.0f;      // largest exponent of a weight by an m that is kept
constexpr float LAG = 8.0f;        // how far, in powers of two, a running maximum may lag
constexpr float NOTHING = -FLT_MAX;   // m of a piece in which a row saw nothing
constexpr int W_COPY = 8, W_MMA = 9, W_FIX = 10, THREADS = 12 * 32;   // warp 11 only gives registers
// Registers of a thread of the softmax groups (eight warps) and of the others (four), out of
// what 12 warps of 168 were launched with.
constexpr int LAUNCH_REGS = 168, SOFTMAX_REGS = 200, OTHER_REGS = 104;
static_assert(8 * SOFTMAX_REGS + 4 * OTHER_REGS <= 12 * LAUNCH_REGS, "more registers than the CTA has would be waited for");
constexpr unsigned long long WAIT_LIMIT_CYCLES = 20000000000ull;   // ~10 s at 2 GHz
constexpr int PLAN_THREADS = 1024;
// Of the plan for at most as many tiles and twice as many requests, whose barriers cost less: us with it and with 1024,
// 64 short prompts 23.2 and 24.8, a 2123-token one 90.6 and 91.8, 64 queries on 32k 63.0 and 65.1.
constexpr int FEW_THREADS = 256;
constexpr int SPLIT_UNITS = 2;     // units per SM below which they may be split

// barriers
enum {
  B_KFULL = 0, B_KFREE = 4, B_VFULL = 8, B_VFREE = 10,   // by panel, by buffer
  B_QFULL = 12, B_QFREE = 14, B_SFULL = 16, B_OFULL = 18,   // by half
  B_PFULL = 20,   // by half, and by half of the block
  B_FIX = 24, B_FIXED = 25, B_DRAIN = 26, N_BAR = 27
};

struct Smem {
  static constexpr int Q = 0, QHALF = 3 * PANEL, K = 2 * QHALF, V = K + K_PANELS * PANEL, VBUF = 2 * PANEL;
  static constexpr int BAR = V + V_BUFS * VBUF, MISC = BAR + 8 * N_BAR, BYTES = (MISC + 16 + 127) / 128 * 128;
  static_assert(BYTES <= 227 * 1024, "shared memory of a CTA");
};
struct Tmem {   // columns; S and O of half t at S + 128 t, O + 128 t
  static constexpr int S = 0, O = 256, COLS = 512;
};

struct Tile {      // rows [row0, row0 + TILE_ROWS) of a request
  int q0, rows;    // the request's first query row and their number
  int row0, kv;    // kv: the request's keys
  int k0, steps;   // its first key row; blocks of 128 keys that the tile's rows see
  long long before;   // steps of a head in the tiles in front of it, a tile with none counted as 1 (SPLIT)
};

struct Share {     // where a CTA's share of the steps begins
  int tile, head, step, pad;
};

struct Header {
  uint32_t status;
  int n_tiles;
  long long share;   // steps of every CTA (SPLIT)
};

// m, l and O of a piece of a unit, as a CTA leaves them: O in the order [DV / 4][row][4]
constexpr int PARTIAL = TILE_ROWS * (DV + 2);   // floats

struct Params {
  const int32_t *cu_q, *cu_kv;
  uint16_t* out;
  float* lse;
  long long out_ld, out_hd;
  Header* header;
  Tile* tiles;
  Share* shares;
  float* partial;   // two for each CTA: of the unit that it continued (0), and of one that it began (1)
  int n_tokens, n_keys, n_req, h, max_tiles, n_ctas, split, bf16;
  uint32_t test_block;   // block of CTA 0 at which the copies stop (DSA_MLA_FLAG_TEST_WAIT_TIMEOUT)
  float scale_log2;      // softmax_scale * log2 e
};

struct Maps {
  CUtensorMap q, k, r, v;
};

// ------------------------------------------------------------------------------ plan
DSA_DEV int clamped(int x, int most) { return min(max(x, 0), most); }

DSA_DEV int rows_of(const Params& P, int r) {
  const int a = clamped(P.cu_q[r], P.n_tokens);
  return max(clamped(P.cu_q[r + 1], P.n_tokens), a) - a;
}

DSA_DEV Tile make_tile(const Params& P, int r, int row0) {
  Tile t;
  t.q0 = clamped(P.cu_q[r], P.n_tokens);
  t.rows = rows_of(P, r);
  t.row0 = row0;
  t.k0 = clamped(P.cu_kv[r], P.n_keys);
  t.kv = max(clamped(P.cu_kv[r + 1], P.n_keys), t.k0) - t.k0;
  const int seen = t.kv - t.rows + min(row0 + TILE_ROWS, t.rows);   // by the tile's last row
  t.steps = (max(seen, 0) + BLOCK - 1) / BLOCK;
  t.before = 0;
  return t;
}

// Exclusive sum of one value a thread over the CTA; `all` becomes the sum.
template <typename T>
DSA_DEV T scan(T v, T* s_warp, T& all) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  T in = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T x = __shfl_up_sync(0xFFFFFFFFu, in, o);
    if (lane >= o) in += x;
  }
  __syncthreads();
  if (lane == 31) s_warp[w] = in;
  __syncthreads();
  T before = in - v;
  all = 0;
  for (int u = 0; u < (int)(blockDim.x >> 5); ++u) {
    if (u < w) before += s_warp[u];
    all += s_warp[u];
  }
  return before;
}

template <int N>   // threads
__global__ void __launch_bounds__(N) plan_kernel(const __grid_constant__ Params P) {
  extern __shared__ int s_tile[];   // [n_req + 1] exclusive prefix of the requests' tiles
  __shared__ int s_warp[N / 32], s_place[N];
  __shared__ long long s_long[N / 32], s_before[N];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = threadIdx.x, n = P.n_req;
  for (int r = tid; r < n; r += N) s_tile[r] = (rows_of(P, r) + TILE_ROWS - 1) / TILE_ROWS;
  __syncthreads();
  const int per = ((n + N - 1) / N) | 1;   // odd: no bank conflicts
  const int r0 = min(tid * per, n), r1 = min(r0 + per, n);
  int mine = 0, all = 0;
  for (int r = r0; r < r1; ++r) mine += s_tile[r];
  int at = scan(mine, s_warp, all);
  for (int r = r0; r < r1; ++r) {
    const int x = s_tile[r];
    s_tile[r] = at;
    at += x;
  }
  if (tid == 0) s_tile[n] = all;
  __syncthreads();
  const int n_tiles = min(all, P.max_tiles);   // ascending cu_q cannot give more
  auto tile = [&](int i) {
    int lo = 0, hi = n;   // the request with s_tile[lo] <= i < s_tile[lo + 1]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (s_tile[mid] <= i) lo = mid; else hi = mid;
    }
    return make_tile(P, lo, (i - s_tile[lo]) * TILE_ROWS);
  };
  long long share = 0;
  if (P.split) {
    // at most a thread for each tile, by the rule of split()
    Tile t = {};
    if (tid < n_tiles) t = tile(tid);
    long long total = 0;
    t.before = scan((long long)(tid < n_tiles ? max(t.steps, 1) : 0), s_long, total);
    if (tid < n_tiles) P.tiles[tid] = t;
    total *= P.h;
    share = max((total + P.n_ctas - 1) / P.n_ctas, 2LL);
    if (tid < n_tiles) s_before[tid] = t.before;
    __syncthreads();
    for (int b = tid; b < P.n_ctas; b += N) {
      const long long at_step = b * share;
      Share s = {-1, 0, 0, 0};
      if (at_step < total) {
        int lo = 0, hi = n_tiles;   // the tile with before[lo] * h <= at_step < before[lo + 1] * h
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (s_before[mid] * P.h <= at_step) lo = mid; else hi = mid;
        }
        const long long steps = ((lo + 1 < n_tiles ? s_before[lo + 1] : total / P.h) - s_before[lo]), rest = at_step - s_before[lo] * P.h;
        s.tile = lo;
        s.head = (int)(rest / steps);
        s.step = (int)(rest - s.head * steps);
      }
      P.shares[b] = s;
    }
  } else {
    // the longest first (all of N - 1 blocks and more alike): a count of each length, the
    // places behind the longer ones, then the tiles.  The order among equal ones changes no result.
    auto place = [](const Tile& t) { return N - 1 - min(t.steps, N - 1); };
    s_place[tid] = 0;
    __syncthreads();
    for (int i = tid; i < n_tiles; i += N) atomicAdd(&s_place[place(tile(i))], 1);
    __syncthreads();
    int total = 0;
    const int before = scan(s_place[tid], s_warp, total);
    __syncthreads();
    s_place[tid] = before;
    __syncthreads();
    for (int i = tid; i < n_tiles; i += N) {
      const Tile t = tile(i);
      P.tiles[atomicAdd(&s_place[place(t)], 1)] = t;
    }
  }
  if (tid == 0) {
    P.header->status = 0;
    P.header->n_tiles = n_tiles;
    P.header->share = share;
  }
}

// ------------------------------------------------------------------------------ shared by the roles
struct Ctx {
  uint32_t sb, bars;
  volatile int* misc;   // [0]: tensor memory address, [1]: abort, [2]: blocks copied,
                        // [3]: block whose values are to be mended
  uint32_t* status;
};

DSA_DEV uint32_t bar(const Ctx& c, int i) { return c.bars + 8u * (uint32_t)i; }
// The waiting part of a bounded wait.  False when the limit passes without a block being copied, or when
// another thread of the CTA has given up.
DSA_DEV bool wait_slow(uint32_t addr, uint32_t parity, volatile int* misc, uint32_t* status) {
  unsigned long long start = clock64();
  int seen = misc[2];
  while (true) {
    if (mbar_wait_susp(addr, parity)) return true;
    if (misc[1]) return false;
    if (misc[2] != seen) {
      seen = misc[2];
      start = clock64();
    }
    if (clock64() - start > WAIT_LIMIT_CYCLES) {
      atomicOr(status, DSA_STATUS_WAIT_TIMEOUT);
      misc[1] = 1;
      return false;
    }
  }
}
DSA_DEV bool wait_1(const Ctx& c, int b, uint32_t parity) {
  const uint32_t addr = bar(c, b);
  return mbar_try(addr, parity) || wait_slow(addr, parity, c.misc, c.status);
}
// The whole warp waits and agrees on the outcome.
DSA_DEV bool wait_w(const Ctx& c, int b, uint32_t parity) {
  const uint32_t addr = bar(c, b);
  const bool ok = mbar_try(addr, parity) || wait_slow(addr, parity, c.misc, c.status);
  return __all_sync(0xFFFFFFFFu, ok);
}
DSA_DEV void arrive_w(const Ctx& c, int b) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar(c, b));
}
// For tests of the failure path: a wait that runs out, after an eighth of the limit.
DSA_DEV bool wait_in_vain(const Ctx& c) {
  const unsigned long long start = clock64();
  while (!mbar_wait_susp(bar(c, B_DRAIN), 0) && clock64() - start < WAIT_LIMIT_CYCLES / 8) {
  }
  atomicOr(c.status, DSA_STATUS_WAIT_TIMEOUT);
  c.misc[1] = 1;
  return false;
}
DSA_DEV bool elect_one() {
  uint32_t e;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
  return e != 0;
}

// A unit, or a CTA's piece of one, as every role sees it.
struct Unit {
  Tile t;
  int head;
  int first[2];    // first row of each half
  bool rows[2];    // whether a half has rows
  int blocks[2];   // blocks of each half in this piece
  bool two;        // SPLIT: the same rows in both halves, which take the piece's blocks in turn
  int s0;          // the piece's first block
  int pieces, part;   // CTAs that share the unit; this piece's partial result

  // whether block i of the piece is half h's, and whether it is the first and the last of these
  DSA_DEV bool has(int h, int i) const { return i < (h == 0 ? blocks[0] : blocks[1]) && (!two || (i & 1) == h); }
  DSA_DEV bool begins(int i) const { return i < (two ? 2 : 1); }
  DSA_DEV bool ends(int h, int i) const { return i + (two ? 2 : 1) >= (h == 0 ? blocks[0] : blocks[1]); }
};

// The units of a CTA, in order.  All roles walk them alike.
template <bool SPLIT>
struct Walk {
  uint32_t round = 0, one = 0;   // one: units of one half so far
  int tile, head, step;          // SPLIT: where the rest of the share begins
  long long left, share;

  DSA_DEV explicit Walk(const Params& P) {
    if (SPLIT) {
      const Share s = P.shares[blockIdx.x];
      tile = s.tile;
      head = s.head;
      step = s.step;
      left = share = P.header->share;
    }
  }
  DSA_DEV bool next(const Params& P, int n_tiles, Unit& x) {
    int i;
    if (SPLIT) {
      if (tile < 0 || left == 0) return false;
      if (head == P.h) {
        head = 0;
        ++tile;
      }
      if (tile >= n_tiles) return false;
      i = tile;
      x.head = head;
    } else {
      const unsigned long long u = (unsigned long long)round * gridDim.x + ((round & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
      ++round;
      if (u >= (unsigned long long)n_tiles * P.h) return false;
      i = (int)(u / (unsigned)P.h);
      x.head = (int)(u - (unsigned long long)i * P.h);
    }
    // plain loads: the plan may be written while this kernel is there already
    const int4* at = reinterpret_cast<const int4*>(P.tiles + i);
    const int4 a = at[0], b = at[1];
    x.t.q0 = a.x; x.t.rows = a.y; x.t.row0 = a.z; x.t.kv = a.w;
    x.t.k0 = b.x; x.t.steps = b.y;
    x.s0 = 0;
    x.pieces = 1;
    x.part = 0;
    int s1 = x.t.steps;
    if (SPLIT) {
      const int steps = max(x.t.steps, 1);
      const long long before = (((long long)(uint32_t)b.w << 32) | (uint32_t)b.z) * P.h + (long long)x.head * steps;
      s1 = (int)min((long long)steps, step + left);
      x.s0 = step;
      x.part = 2 * blockIdx.x + (step == 0 ? 1 : 0);
      x.pieces = (int)((before + steps - 1) / share - before / share) + 1;
      left -= s1 - step;
      step = 0;
      ++head;
    }
    const int left_rows = x.t.rows - x.t.row0;
    x.two = SPLIT && left_rows <= 128 && x.pieces > 1;
    const bool second = left_rows <= 128 && !x.two && (one++ & 1);
    const bool both = left_rows > 128 || x.two;
    x.rows[0] = both || !second;
    x.rows[1] = both || second;
    x.first[0] = x.t.row0;
    x.first[1] = x.t.row0 + (left_rows > 128 ? 128 : 0);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int seen = x.t.kv - x.t.rows + min(x.first[h] + 128, x.t.rows);   // by the half's last row
      x.blocks[h] = x.rows[h] ? min(max((max(seen, 0) + BLOCK - 1) / BLOCK - x.s0, 0), s1 - x.s0) : 0;
    }
    return true;
  }
};

// ------------------------------------------------------------------------------ copies
DSA_DEV void expect(uint32_t b, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.release.cta.shared::cta.b64 _, [%0], %1;" ::"r"(b), "r"(bytes) : "memory");
}
DSA_DEV void tma3(uint32_t dst, const CUtensorMap* map, int c0, int c1, int c2, uint32_t b) {
  asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
               "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(b)
               : "memory");
}
DSA_DEV void tma2(uint32_t dst, const CUtensorMap* map, int c0, int c1, uint32_t b) {
  asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
               "l"(map), "r"(c0), "r"(c1), "r"(b)
               : "memory");
}

// In the order in which the products take them: a block's keys, and its values in front of the next
// block's keys.
template <bool SPLIT>
DSA_DEV void copies(const Params& P, const Maps& M, const Ctx& c, int n_tiles) {
  const bool one = elect_one();
  uint32_t g = 0, kp = 0, nq[2] = {0, 0};   // blocks, panels of keys, units of each half
  int v_row = 0, v_head = 0;
  bool v_due = false, ok = true;
  auto values = [&](uint32_t i) {   // of block i
    const int buf = i % V_BUFS;
    if (!wait_w(c, B_VFREE + buf, ((i / V_BUFS) & 1) ^ 1)) return false;
    if (one) {
      const uint32_t to = c.sb + Smem::V + buf * Smem::VBUF, b = bar(c, B_VFULL + buf);
      expect(b, Smem::VBUF);
      tma3(to, &M.v, 0, v_head, v_row, b);
      tma3(to + PANEL, &M.v, 64, v_head, v_row, b);
    }
    return true;
  };
  Walk<SPLIT> walk(P);
  Unit x;
  while (ok && walk.next(P, n_tiles, x)) {
    const int blocks = max(x.blocks[0], x.blocks[1]);
    for (int i = 0; ok && i < blocks; ++i, ++g) {
      if (g == P.test_block && blockIdx.x == 0) {
        ok = wait_in_vain(c);
        break;
      }
      if (v_due && !(ok = values(g - 1))) break;
      v_due = false;
      const int row = x.t.k0 + (x.s0 + i) * BLOCK;
      if (i == 0) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (ok && x.has(h, x.two ? h : 0)) {
            ok = wait_w(c, B_QFREE + h, (nq[h] & 1) ^ 1);
            if (!ok) break;
            ++nq[h];
            if (one) {
              expect(bar(c, B_QFULL + h), Smem::QHALF);
#pragma unroll
              for (int p = 0; p < 3; ++p)
                tma3(c.sb + Smem::Q + h * Smem::QHALF + p * PANEL, &M.q, 64 * p, x.head, x.t.q0 + x.first[h], bar(c, B_QFULL + h));
            }
          }
      }
#pragma unroll
      for (int p = 0; p < 3; ++p) {
        const int slot = kp % K_PANELS;
        if (!ok || !(ok = wait_w(c, B_KFREE + slot, ((kp / K_PANELS) & 1) ^ 1))) break;
        if (one) {
          const uint32_t to = c.sb + Smem::K + slot * PANEL, b = bar(c, B_KFULL + slot);
          expect(b, PANEL);
          if (p < 2) tma3(to, &M.k, 64 * p, x.head, row, b);
          else tma2(to, &M.r, 0, row, b);
        }
        ++kp;
      }
      if (!ok) break;
      v_row = row;
      v_head = x.head;
      v_due = true;
      if (one) c.misc[2] = (int)g;
    }
  }
  if (ok && v_due) ok = values(g - 1);
  if (!ok) {
    // gave up: wait, with a limit, for the copies in flight.  A buffer's last copy is that of its last
    // use; an older phase's parity can only end this wait early where a newer copy was not issued.
    const unsigned long long start = clock64();
    auto settle = [&](int b, uint32_t uses) {   // uses: phases that were begun
      while (uses > 0 && !mbar_wait_susp(bar(c, b), (uses - 1) & 1) && clock64() - start < WAIT_LIMIT_CYCLES / 8) {
      }
    };
    for (int s = 0; s < K_PANELS; ++s) settle(B_KFULL + s, (kp + K_PANELS - 1 - s) / K_PANELS);
    for (int h = 0; h < 2; ++h) settle(B_QFULL + h, nq[h]);
    // values were asked for of the blocks up to g - 1, or g - 2
    const uint32_t nv = v_due ? (g > 0 ? g - 1 : 0) : g;
    for (int s = 0; s < V_BUFS; ++s) settle(B_VFULL + s, (nv + V_BUFS - 1 - s) / V_BUFS);
  }
}

// ------------------------------------------------------------------------------ products
// One thread runs this role.  (The whole warp with an elected lane to issue, and votes on each wait,
// took 5700 cycles for a block of both halves, whose products are 2560: the softmax, 1400 a half, was
// waiting for the next instruction to be issued.)
template <bool SPLIT>
DSA_DEV void products(const Params& P, const Ctx& c, uint32_t tmem, int n_tiles) {
  const uint32_t type = P.bf16 ? (1u << 7) | (1u << 10) : 0u;
  const uint32_t ID_QK = idesc_f16(128, BLOCK, 0, 0) | type, ID_PV = idesc_f16(128, DV, 0, 1) | type;
  const uint64_t d_q = sdesc(c.sb + Smem::Q, 16, 1024);
  const uint64_t d_k = sdesc(c.sb + Smem::K, 16, 1024);
  const uint64_t d_v = sdesc(c.sb + Smem::V, PANEL, 1024);
  // bits of the halves: whether weights are due, the block at hand is its unit's last one in the half, and parities
  uint32_t g = 0, kp = 0, fixes = 0, due = 0, last = 0, p_parity = 0, q_parity = 0;
  bool first = false, partial = false;   // of the block whose weights are due; partial: it has rows that are not the request's
  Walk<SPLIT> walk(P);
  Unit x;
  int i = 0, blocks = 0;
  while (true) {
    bool more = true;
    while (i == blocks && more) {
      more = walk.next(P, n_tiles, x);
      blocks = more ? max(x.blocks[0], x.blocks[1]) : 0;
      i = 0;
    }
    if (!more && due == 0) return;
    const uint32_t now = more ? (x.has(0, i) ? 1u : 0u) | (x.has(1, i) ? 2u : 0u) : 0u;
    const uint32_t ends = more ? now & ((x.ends(0, i) ? 1u : 0u) | (x.ends(1, i) ? 2u : 0u)) : 0u;
    const uint32_t due_at_first = due;
    bool v_there = false, k_there = false;
    // a half's scores follow its weights' product with the block before; a half alone goes first, so that its scores
    // are under way while the other's weights are waited for
#pragma unroll 1
    for (int t = 0; t < 2; ++t) {
      const uint32_t h = now == 2u ? 1 - t : t, bit = 1u << h;
      if (due & bit) {   // O += P V with block g - 1
        const uint32_t buf = (g - 1) % V_BUFS;
        if (!v_there) {
          if (partial) {
            if (!wait_1(c, B_FIXED, fixes & 1)) return;
            ++fixes;
          } else if (!wait_1(c, B_VFULL + buf, ((g - 1) / V_BUFS) & 1)) {
            return;
          }
          v_there = true;
        }
        const uint64_t v = d_v + ((buf * Smem::VBUF) >> 4);
#pragma unroll
        for (int part = 0; part < 2; ++part) {
          if (!wait_1(c, B_PFULL + 2 * h + part, (p_parity >> h) & 1)) return;
          tc_fence_after();
#pragma unroll
          for (int k = 4 * part; k < 4 * part + 4; ++k)
            mma_ts(tmem + Tmem::O + 128 * h, tmem + Tmem::S + 128 * h + 8 * k, v + (k * 2048 >> 4), ID_PV, k > 0 || !first ? 1u : 0u);
        }
        p_parity ^= bit;
        if (last & bit) tc_commit(bar(c, B_OFULL + h));
      }
      if (now & bit) {   // S of block g
        if (x.begins(i)) {
          if (!wait_1(c, B_QFULL + h, (q_parity >> h) & 1)) return;
          q_parity ^= bit;
        }
        tc_fence_after();   // the scores before were read
        const bool k_last = (now >> 1) == h || now == 1u;   // the last half that reads the keys
        const uint64_t q = d_q + ((h * Smem::QHALF) >> 4);
#pragma unroll
        for (int p = 0; p < 3; ++p) {
          const uint32_t slot = (kp + p) % K_PANELS;
          if (!k_there && !wait_1(c, B_KFULL + slot, ((kp + p) / K_PANELS) & 1)) return;
          const uint64_t k_at = d_k + ((slot * PANEL) >> 4);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma_ss(tmem + Tmem::S + 128 * h, q + ((p * PANEL + k * 32) >> 4), k_at + (k * 32 >> 4), ID_QK, (p > 0 || k > 0) ? 1u : 0u);
          if (k_last) tc_commit(bar(c, B_KFREE + slot));
        }
        k_there = true;
        if (ends & bit) tc_commit(bar(c, B_QFREE + h));
        tc_commit(bar(c, B_SFULL + h));
      }
    }
    if (due_at_first) tc_commit(bar(c, B_VFREE + (g - 1) % V_BUFS));
    if (!more) return;
    due = now;
    first = x.begins(i);
    last = ends;
    partial = x.t.kv - (x.s0 + i) * BLOCK < BLOCK;
    if (partial) {   // its values are mended while its weights are formed
      c.misc[3] = (int)g;
      mbar_arrive(bar(c, B_FIX));
    }
    kp += 3;
    ++i;
    ++g;
  }
}

// The values of a request's last block: rows that are not the request's may hold anything, and 0 * NaN is
// not 0.  One warp, for each block that the products name: those of the blocks two before it were used by
// then, so that its wait for them is for the phase that comes next.
template <bool SPLIT>
DSA_DEV void fix_values(const Params& P, const Ctx& c, uint8_t* sm, int n_tiles) {
  const int lane = threadIdx.x & 31;
  uint32_t fixes = 0;
  Walk<SPLIT> walk(P);
  Unit x;
  while (walk.next(P, n_tiles, x)) {
    const int blocks = max(x.blocks[0], x.blocks[1]), rows = x.t.kv - (x.s0 + blocks - 1) * BLOCK;
    if (blocks == 0 || rows >= BLOCK) continue;   // only the last block can have fewer
    if (!wait_w(c, B_FIX, fixes & 1)) return;
    ++fixes;
    const uint32_t g = (uint32_t)c.misc[3];
    if (!wait_w(c, B_VFULL + g % V_BUFS, (g / V_BUFS) & 1)) return;
    uint8_t* v = sm + Smem::V + g % V_BUFS * Smem::VBUF;
    for (int r = rows + (lane >> 3); r < BLOCK; r += 4) {
      *reinterpret_cast<uint4*>(v + r * 128 + (lane & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
      *reinterpret_cast<uint4*>(v + PANEL + r * 128 + (lane & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
    }
    fence_async_smem();
    arrive_w(c, B_FIXED);
  }
}

// ------------------------------------------------------------------------------ softmax
DSA_DEV float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
DSA_DEV uint64_t pair(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
// two fp32 operations in one instruction
DSA_DEV void fma2(uint32_t& x0, uint32_t& x1, uint64_t mul, uint64_t add) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "r"(x0), "r"(x1));
  asm("fma.rn.f32x2 %0, %0, %1, %2;" : "+l"(v) : "l"(mul), "l"(add));
  asm("mov.b64 {%0, %1}, %2;" : "=r"(x0), "=r"(x1) : "l"(v));
}
DSA_DEV void add2(float& s0, float& s1, float a, float b) {
  uint64_t v = pair(s0, s1);
  asm("add.rn.f32x2 %0, %0, %1;" : "+l"(v) : "l"(pair(a, b)));
  asm("mov.b64 {%0, %1}, %2;" : "=f"(s0), "=f"(s1) : "l"(v));
}
DSA_DEV float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
template <bool BF16>
DSA_DEV uint32_t pack(float a, float b) {
  if (!BF16) return pack_f16x2(a, b);
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}
template <bool BF16>
DSA_DEV float2 unpack(uint32_t w) {
  if (!BF16) return __half22float2(*reinterpret_cast<const __half2*>(&w));
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
// The sum of a row at position pos.  Weights are 1 and more at their largest, so that one of 0 has seen nothing; but for a row
// that has keys, all of whose scores are -inf: its query is not finite, and the softmax not defined.
DSA_DEV float defined(float sum, int pos) { return sum == 0.f && pos >= 0 ? __int_as_float(0x7FC00000) : sum; }
// 1 / sum; 0 for a row that saw nothing, and a NaN stays one
DSA_DEV float inverse(float sum) { return sum > 0.f ? 1.0f / sum : (sum == 0.f ? 0.f : sum); }
DSA_DEV float lse_of(float m, float l) { return l == 0.f ? -INFINITY : 0.6931471805599453f * (m + log2f(l)); }

template <bool BF16, bool SPLIT>
DSA_DEV void softmax(const Params& P, const Ctx& c, uint32_t tmem, int n_tiles, int h) {
  const int row_in = threadIdx.x & 127;
  const uint32_t lanes = (uint32_t)((threadIdx.x >> 5) & 3) << 21;   // the warp's 32 lanes of tensor memory
  const uint32_t ts = tmem + lanes + Tmem::S + 128 * h, to = tmem + lanes + Tmem::O + 128 * h;
  uint32_t ns = 0, no = 0;
  Walk<SPLIT> walk(P);
  Unit x;
  while (walk.next(P, n_tiles, x)) {
    if (!(h == 0 ? x.rows[0] : x.rows[1])) continue;
    const int blocks = h == 0 ? x.blocks[0] : x.blocks[1], first = h == 0 ? x.first[0] : x.first[1];
    const int begin = x.two ? h : 0, stride = x.two ? 2 : 1;
    const int row = first + row_in;
    const bool live = row < x.t.rows;
    const int pos0 = x.t.kv - x.t.rows, pos = pos0 + min(row, x.t.rows - 1);
    const uint64_t mul = pair(P.scale_log2, P.scale_log2);
    float m = 0.f, l = 0.f;
    bool fresh = true;   // m is not set: every score so far was masked
    for (int i = begin; i < blocks; i += stride) {
      const int base = (x.s0 + i) * BLOCK;
      if (!wait_w(c, B_SFULL + h, ns & 1)) return;
      ++ns;
      tc_fence_after();
      uint32_t x2[128];
#pragma unroll
      for (int k = 0; k < 128; k += 32) tmem_ld32(ts + k, *reinterpret_cast<uint32_t(*)[32]>(x2 + k));
      const uint64_t add = pair(-m, -m);
      tc_wait_ld();
#pragma unroll
      for (int e = 0; e < 128; e += 2) fma2(x2[e], x2[e + 1], mul, add);
      if (base + BLOCK - 1 > pos0 + first) {   // the half's first row sees less
        const int last = pos - base;
#pragma unroll
        for (int e = 0; e < 128; ++e)
          if (e > last) x2[e] = 0xFF800000u;   // -inf
      }
      float t4[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        t4[q] = fmaxf(__uint_as_float(x2[q]), __uint_as_float(x2[q + 4]));
#pragma unroll
        for (int e = 8; e < 128; e += 8) t4[q] = max3(t4[q], __uint_as_float(x2[e + q]), __uint_as_float(x2[e + 4 + q]));
      }
      const float top = fmaxf(max3(t4[0], t4[1], t4[2]), t4[3]);
      if (__any_sync(0xFFFFFFFFu, fresh || top > MOST)) {
        const bool up = top > (fresh ? -INFINITY : LAG);
        // by delta, not by m's rounded step: from 2^23 on m + delta is rounded
        const float delta = up ? (fresh ? top : floorf(top)) : 0.f;
        const float f = (up && !fresh) ? ex2(-delta) : 1.0f;
        if (up) fresh = false;
        m += delta;
        l *= f;
#pragma unroll
        for (int e = 0; e < 128; ++e) x2[e] = __float_as_uint(__uint_as_float(x2[e]) - delta);
        if (i > begin && __any_sync(0xFFFFFFFFu, f != 1.0f)) {
          // the product of the block before is done: these scores were issued after it
#pragma unroll 1
          for (int k = 0; k < DV; k += 8) {
            uint32_t o[8];
            tmem_ld8(to + k, o);
            tc_wait_ld();
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
            tmem_st8(to + k, o);
          }
        }
      }
#pragma unroll
      for (int part = 0; part < 2; ++part) {   // the products begin with the first 64 keys
        uint32_t p[32];
        float s0 = 0.f, s1 = 0.f, s2 = 0.f, s3 = 0.f;
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
          const uint32_t* u = x2 + 64 * part + 2 * e;
          const float w0 = ex2(__uint_as_float(u[0])), w1 = ex2(__uint_as_float(u[1]));
          const float w2 = ex2(__uint_as_float(u[2])), w3 = ex2(__uint_as_float(u[3]));
          add2(s0, s1, w0, w1);
          add2(s2, s3, w2, w3);
          p[e] = pack<BF16>(w0, w1);
          p[e + 1] = pack<BF16>(w2, w3);
        }
        l += (s0 + s1) + (s2 + s3);
        tmem_st32(ts + 32 * part, p);
        tc_wait_st();
        tc_fence_before();
        arrive_w(c, B_PFULL + 2 * h + part);
      }
    }
    // ---- result
    const bool some = blocks > begin;
    if (some) {
      if (!wait_w(c, B_OFULL + h, no & 1)) return;
      ++no;
      tc_fence_after();
    }
    const long long token = (long long)x.t.q0 + row;
    if (!SPLIT || x.pieces == 1) {
      l = defined(l, pos);
      uint16_t* dst = P.out + token * P.out_ld + x.head * P.out_hd;
      const bool wide = ((uintptr_t)dst & 31) == 0;
      const float inv = inverse(l);
#pragma unroll 1
      for (int k = 0; k < DV; k += 32) {
        uint32_t o[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] = 0u;
        if (some) {
          tmem_ld32(to + k, o);
          tc_wait_ld();
        }
        if (live) {
#pragma unroll
          for (int e = 0; e < 32; e += 16) {
            uint32_t v[8];
#pragma unroll
            for (int q = 0; q < 8; ++q)
              v[q] = pack<BF16>(__uint_as_float(o[e + 2 * q]) * inv, __uint_as_float(o[e + 2 * q + 1]) * inv);
            // a lane for a row touches 32 lines with every store: the fewer the better
            if (wide) {
              stg256(dst + k + e, v);
            } else {
              *reinterpret_cast<uint4*>(dst + k + e) = make_uint4(v[0], v[1], v[2], v[3]);
              *reinterpret_cast<uint4*>(dst + k + e + 8) = make_uint4(v[4], v[5], v[6], v[7]);
            }
          }
        }
      }
      if (live && P.lse) P.lse[token * P.h + x.head] = lse_of(m, l);
    } else {
      float* at = P.partial + (long long)x.part * PARTIAL;
      const int r = row - x.t.row0 + (x.two ? 128 * h : 0);
      if (some) {
#pragma unroll 1
        for (int k = 0; k < DV; k += 32) {
          uint32_t o[32];
          tmem_ld32(to + k, o);
          tc_wait_ld();
          if (live) {
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              *reinterpret_cast<uint4*>(at + ((k + e) / 4 * TILE_ROWS + r) * 4) = make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
          }
        }
      }
      if (live) {
        at[TILE_ROWS * DV + r] = fresh && !(l != l) ? NOTHING : m;
        at[TILE_ROWS * (DV + 1) + r] = l;
      }
    }
    tc_fence_before();   // O was read, before the next unit's products
  }
}

template <bool BF16, bool SPLIT>
__global__ void __launch_bounds__(THREADS, 1) mla_kernel(const __grid_constant__ Params P, const __grid_constant__ Maps M) {
  extern __shared__ __align__(1024) uint8_t smem[];
  Ctx c;
  c.sb = smem_u32(smem);
  c.bars = c.sb + Smem::BAR;
  c.misc = reinterpret_cast<volatile int*>(smem + Smem::MISC);
  c.status = &P.header->status;
  const int warp = threadIdx.x >> 5;
  if (SPLIT) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // the join
  if (threadIdx.x == 0) {
    for (int i = 0; i < N_BAR; ++i) mbar_init(bar(c, i), i >= B_PFULL && i < B_PFULL + 4 ? 4 : 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    c.misc[1] = c.misc[2] = 0;
  }
  if (warp == W_MMA) tmem_alloc(c.sb + Smem::MISC, Tmem::COLS);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = (uint32_t)c.misc[0];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int n_tiles = P.header->n_tiles;
  if (warp < W_COPY) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(SOFTMAX_REGS));
    softmax<BF16, SPLIT>(P, c, tmem, n_tiles, warp >> 2);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(OTHER_REGS));
    if (warp == W_COPY) copies<SPLIT>(P, M, c, n_tiles);
    else if (warp == W_FIX) fix_values<SPLIT>(P, c, smem, n_tiles);
    else if (warp == W_MMA && elect_one()) products<SPLIT>(P, c, tmem, n_tiles);
  }
  __syncwarp();
  if (warp == W_MMA) {
    if (elect_one()) tc_commit(bar(c, B_DRAIN));
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == W_MMA && (threadIdx.x & 31) == 0) {
    // every product has completed before tensor memory is released
    const unsigned long long start = clock64();
    while (!mbar_wait_susp(bar(c, B_DRAIN), 0) && clock64() - start < WAIT_LIMIT_CYCLES) {
    }
  }
  __syncthreads();
  if (warp == W_MMA) {
    tc_fence_after();
    tmem_dealloc(tmem, Tmem::COLS);
  }
}

// ------------------------------------------------------------------------------ join
// Units in several pieces, 32 rows and 32 dims at a time: a warp has 4 of the dims, a lane a row.  The
// pieces are joined in their order, AT_ONCE of them on their way together.
constexpr int JOIN_THREADS = 256, AT_ONCE = 8;
template <bool BF16>
__global__ void __launch_bounds__(JOIN_THREADS) join_kernel(const __grid_constant__ Params P) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  constexpr int ROWS = TILE_ROWS / 32, PARTS = ROWS * (DV / 32);
  const int n_tiles = P.header->n_tiles, lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const long long share = P.header->share;
  const int items = n_tiles * P.h * PARTS;
  for (int item = blockIdx.x; item < items; item += gridDim.x) {
    const int unit = item / PARTS, i = unit / P.h, head = unit - i * P.h;
    const Tile t = P.tiles[i];
    const long long steps = max(t.steps, 1), before = t.before * P.h + head * steps;
    const int b0 = (int)(before / share), b1 = (int)((before + steps - 1) / share);
    const int r = (item % ROWS) * 32 + lane, row = t.row0 + r, chunk = item % PARTS / ROWS * 8 + w;
    if (b0 == b1 || row >= t.rows) continue;
    const int halves = t.rows - t.row0 <= 128 ? 2 : 1;   // 2: both halves had these rows
    const int n = (b1 - b0 + 1) * halves;
    float m = NOTHING, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
    for (int j0 = 0; j0 < n; j0 += AT_ONCE) {
      float pm[AT_ONCE], pl[AT_ONCE];
      float4 po[AT_ONCE];
#pragma unroll
      for (int j = 0; j < AT_ONCE; ++j) {
        pm[j] = NOTHING;
        pl[j] = 0.f;
        po[j] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (j0 + j < n) {
          const int b = b0 + (j0 + j) / halves;
          const int at_row = r + (j0 + j) % halves * 128;
          const float* at = P.partial + (2LL * b + (b == b0 ? 1 : 0)) * PARTIAL;
          pm[j] = at[TILE_ROWS * DV + at_row];
          pl[j] = at[TILE_ROWS * (DV + 1) + at_row];
          po[j] = *reinterpret_cast<const float4*>(at + (chunk * TILE_ROWS + at_row) * 4);
        }
      }
      float top = m;
#pragma unroll
      for (int j = 0; j < AT_ONCE; ++j) top = fmaxf(top, pm[j]);
      const float f0 = ex2(m - top);
      l *= f0;
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] *= f0;
#pragma unroll
      for (int j = 0; j < AT_ONCE; ++j) {
        if (pm[j] == NOTHING) continue;   // O is not written
        const float f = ex2(pm[j] - top);
        l = fmaf(pl[j], f, l);
        o[0] = fmaf(po[j].x, f, o[0]);
        o[1] = fmaf(po[j].y, f, o[1]);
        o[2] = fmaf(po[j].z, f, o[2]);
        o[3] = fmaf(po[j].w, f, o[3]);
      }
      m = top;
    }
    const long long token = (long long)t.q0 + row;
    l = defined(l, t.kv - t.rows + row);
    const float inv = inverse(l);
    *reinterpret_cast<uint2*>(P.out + token * P.out_ld + head * P.out_hd + 4 * chunk) =
        make_uint2(pack<BF16>(o[0] * inv, o[1] * inv), pack<BF16>(o[2] * inv, o[3] * inv));
    if (chunk == 0 && P.lse) P.lse[token * P.h + head] = lse_of(m, l);
  }
}

// ------------------------------------------------------------------------------ host
static bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

static int check(const dsa_mla_params* p) {
  if (!p || p->n_tokens < 0 || p->n_keys < 0 || p->n_req < 0 || p->h < 1 || p->max_q_len < 0 || p->max_kv_len < 0 ||
      (p->type != DSA_MLA_BF16 && p->type != DSA_MLA_FP16) || !isfinite(p->softmax_scale) ||
      (p->flags & ~DSA_MLA_FLAG_TEST_WAIT_TIMEOUT) != 0)
    return DSA_ERR_INVALID_ARG;
  if (p->n_tokens > (1 << 30) || p->n_keys > (1 << 30) || p->n_req > DSA_MLA_MAX_REQ || p->h > DSA_MLA_MAX_HEADS)
    return DSA_ERR_UNSUPPORTED_SHAPE;
  return DSA_OK;
}

struct Layout {
  int max_tiles;
  bool split;
  size_t shares, tiles, partial, bytes;
};

static size_t up(size_t x) { return (x + 255) / 256 * 256; }

static Layout layout(const dsa_mla_params* p, int sms) {
  Layout L;
  // ascending cu_q cannot give more
  L.max_tiles = (int)(((long long)p->n_tokens + (TILE_ROWS - 1LL) * p->n_req) / TILE_ROWS);
  // Whether units may be split, by the most tiles that the requests are expected to have.  The plan
  // has a thread for each tile then.
  long long tiles = (long long)p->n_req * ((p->max_q_len + (long long)TILE_ROWS - 1) / TILE_ROWS);
  if (tiles > L.max_tiles) tiles = L.max_tiles;
  L.split = tiles * p->h < SPLIT_UNITS * (long long)sms && p->max_kv_len > 2 * BLOCK && L.max_tiles <= PLAN_THREADS;
  size_t at = 256;
  L.shares = at;
  at += up(sms * sizeof(Share));
  L.tiles = at;
  at += up((size_t)L.max_tiles * sizeof(Tile));
  L.partial = at;
  if (L.split) at += up((size_t)sms * 2 * PARTIAL * sizeof(float));
  L.bytes = at;
  return L;
}

typedef CUresult (*EncodeFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                             const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                             CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The driver's function that describes a tensor to the copy engine: looked up once.
static EncodeFn encode_fn() {
  static std::atomic<void*> known{nullptr};
  void* fn = known.load(std::memory_order_acquire);
  if (!fn) {
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess)
      return nullptr;
    known.store(fn, std::memory_order_release);
  }
  return reinterpret_cast<EncodeFn>(fn);
}

// [n][h][d] values of 2 bytes, copied in panels of 64 dims x 128 rows of one head
static bool describe(CUtensorMap* map, EncodeFn fn, int bf16, const void* x, int d, int h, int n, int64_t ld, int64_t hd) {
  const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)h, (cuuint64_t)n};
  const cuuint64_t pitch[2] = {(cuuint64_t)hd * 2, (cuuint64_t)ld * 2};
  const cuuint32_t box[3] = {64, 1, 128}, ones[3] = {1, 1, 1};
  return fn(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void*>(x), dims,
            pitch, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
static bool describe_rope(CUtensorMap* map, EncodeFn fn, int bf16, const void* x, int n, int64_t ld) {
  const cuuint64_t dims[2] = {DR, (cuuint64_t)n};
  const cuuint64_t pitch[1] = {(cuuint64_t)ld * 2};
  const cuuint32_t box[2] = {64, 128}, ones[2] = {1, 1};
  return fn(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, const_cast<void*>(x), dims,
            pitch, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

static cudaError_t set_smem(const void* kernel, int bytes) {
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

template <bool BF16, bool SPLIT>
static int launch(const Params& P, const Maps& M, cudaStream_t st) {
  // the kernel's groups trade the registers that its launch gave them
  cudaFuncAttributes a;
  if (cudaFuncGetAttributes(&a, mla_kernel<BF16, SPLIT>) != cudaSuccess || a.numRegs != LAUNCH_REGS) return DSA_ERR_CUDA;
  if (set_smem((const void*)mla_kernel<BF16, SPLIT>, Smem::BYTES) != cudaSuccess) return DSA_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3((unsigned)P.n_ctas);
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = Smem::BYTES;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, mla_kernel<BF16, SPLIT>, P, M) != cudaSuccess) return DSA_ERR_CUDA;
  if (!SPLIT) return DSA_OK;
  cfg.gridDim = dim3((unsigned)P.n_ctas * 4);
  cfg.blockDim = dim3(JOIN_THREADS);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, join_kernel<BF16>, P) == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}

}  // namespace dsa_mla

extern "C" {

int dsa_mla_params_init(dsa_mla_params* p, int32_t n_tokens, int32_t n_keys, int32_t n_req, int32_t h) {
  if (!p) return DSA_ERR_INVALID_ARG;
  p->n_tokens = n_tokens;
  p->n_keys = n_keys;
  p->n_req = n_req;
  p->h = h;
  p->max_q_len = n_tokens;
  p->max_kv_len = n_keys;
  p->type = DSA_MLA_BF16;
  p->softmax_scale = (float)(1.0 / sqrt(192.0));
  p->flags = 0;
  return dsa_mla::check(p);
}

size_t dsa_mla_prefill_workspace_size(const dsa_mla_params* p, int num_sms) {
  if (dsa_mla::check(p) != DSA_OK) return 0;
  if (num_sms <= 0 && dsa::current_sms(&num_sms) != DSA_OK) return 0;
  return dsa_mla::layout(p, num_sms).bytes;
}

int dsa_mla_prefill_fwd(const void* q, int64_t q_ld, int64_t q_hd, const void* k_nope, int64_t k_ld, int64_t k_hd,
                        const void* k_rope, int64_t k_rope_ld, const void* v, int64_t v_ld, int64_t v_hd,
                        const int32_t* cu_q, const int32_t* cu_kv, void* out, int64_t out_ld, int64_t out_hd, float* lse,
                        const dsa_mla_params* p, void* workspace, size_t workspace_bytes, void* stream) {
  using namespace dsa_mla;
  const int rc = check(p);
  if (rc != DSA_OK) return rc;
  if (!workspace || !aligned(workspace, 256)) return DSA_ERR_INVALID_ARG;
  const bool empty = p->n_tokens == 0 || p->n_req == 0;
  auto bad = [&](const void* x, int64_t ld, int64_t hd, int d, int n) {
    return !x || !aligned(x, 16) || ld % 8 != 0 || hd % 8 != 0 || ld < 0 || hd < 0 || ld >= (1LL << 37) || hd >= (1LL << 37) ||
           (n > 1 && ld < d) || (p->h > 1 && hd < d);
  };
  if (!empty) {
    if (bad(q, q_ld, q_hd, DQ, p->n_tokens) || bad(out, out_ld, out_hd, DV, p->n_tokens) || !cu_q || !cu_kv || !aligned(cu_q, 4) ||
        !aligned(cu_kv, 4) || !aligned(lse, 4))
      return DSA_ERR_INVALID_ARG;
    if (p->n_keys > 0 && (bad(k_nope, k_ld, k_hd, DN, p->n_keys) || bad(v, v_ld, v_hd, DV, p->n_keys) || !k_rope ||
                          !aligned(k_rope, 16) || k_rope_ld % 8 != 0 || k_rope_ld < 0 || k_rope_ld >= (1LL << 37) ||
                          (p->n_keys > 1 && k_rope_ld < DR)))
      return DSA_ERR_INVALID_ARG;
  }
  int sms = 0;
  const int device_rc = dsa::gb300_sms(&sms);
  if (device_rc != DSA_OK) return device_rc;
  const Layout L = layout(p, sms);
  if (workspace_bytes < L.bytes) return DSA_ERR_WORKSPACE_TOO_SMALL;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  cudaStream_t st = (cudaStream_t)stream;
  if (empty) return cudaMemsetAsync(ws, 0, sizeof(uint32_t), st) == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
  Params P;
  P.cu_q = cu_q;
  P.cu_kv = cu_kv;
  P.out = static_cast<uint16_t*>(out);
  P.lse = lse;
  P.out_ld = out_ld;
  P.out_hd = out_hd;
  P.header = reinterpret_cast<Header*>(ws);
  P.shares = reinterpret_cast<Share*>(ws + L.shares);
  P.tiles = reinterpret_cast<Tile*>(ws + L.tiles);
  P.partial = reinterpret_cast<float*>(ws + L.partial);
  P.n_tokens = p->n_tokens;
  P.n_keys = p->n_keys;
  P.n_req = p->n_req;
  P.h = p->h;
  P.max_tiles = L.max_tiles;
  P.n_ctas = sms;
  P.split = L.split;
  P.bf16 = p->type == DSA_MLA_BF16;
  P.test_block = p->flags & DSA_MLA_FLAG_TEST_WAIT_TIMEOUT ? 1u : 0xFFFFFFFFu;
  P.scale_log2 = p->softmax_scale * 1.4426950408889634f;
  Maps M = {};
  const EncodeFn fn = encode_fn();
  if (!fn) return DSA_ERR_CUDA;
  // a pitch that no second row or head uses may be anything: the copies are given a dense one
  auto pitch = [](int64_t x, int64_t dense, int n) { return n > 1 ? x : dense; };
  if (!describe(&M.q, fn, P.bf16, q, DQ, P.h, P.n_tokens, pitch(q_ld, (int64_t)P.h * DQ, P.n_tokens), pitch(q_hd, DQ, P.h)))
    return DSA_ERR_CUDA;
  // without keys no unit has blocks, and these are not used
  if (P.n_keys > 0 &&
      (!describe(&M.k, fn, P.bf16, k_nope, DN, P.h, P.n_keys, pitch(k_ld, (int64_t)P.h * DN, P.n_keys), pitch(k_hd, DN, P.h)) ||
       !describe(&M.v, fn, P.bf16, v, DV, P.h, P.n_keys, pitch(v_ld, (int64_t)P.h * DV, P.n_keys), pitch(v_hd, DV, P.h)) ||
       !describe_rope(&M.r, fn, P.bf16, k_rope, P.n_keys, pitch(k_rope_ld, DR, P.n_keys))))
    return DSA_ERR_CUDA;
  const size_t smem = (size_t)(P.n_req + 1) * sizeof(int);
  static_assert((DSA_MLA_MAX_REQ + 1) * sizeof(int) <= 34 * 1024, "the plan's dynamic shared memory needs no permission");
  if (P.max_tiles <= FEW_THREADS && P.n_req <= 2 * FEW_THREADS) plan_kernel<FEW_THREADS><<<1, FEW_THREADS, smem, st>>>(P);
  else plan_kernel<PLAN_THREADS><<<1, PLAN_THREADS, smem, st>>>(P);
  if (cudaGetLastError() != cudaSuccess) return DSA_ERR_CUDA;
  if (P.bf16) return P.split ? launch<true, true>(P, M, st) : launch<true, false>(P, M, st);
  return P.split ? launch<false, true>(P, M, st) : launch<false, false>(P, M, st);
}

}  // extern "C"
