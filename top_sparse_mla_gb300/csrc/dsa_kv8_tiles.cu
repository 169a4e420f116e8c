// Attention over the paged 8-bit cache for requests with many query rows (prefill): tiles
// of 256 rows on the tensor cores (tcgen05), as dsa_kv8_attn.cu's plan lists them.
//
// One persistent CTA per SM takes units (tile, KV head).  Roles:
//   - warps 0-3 and 4-7, a softmax group for each half of the tile (128 rows): a thread
//     owns a query row.  It scales its row to fp16 into shared memory, and for each block
//     of 128 cached tokens reads its scores from tensor memory, forms the weights and
//     writes them back as fp16 over the scores; in the end it divides its row of O by the
//     softmax's sum and stores it.
//   - warp 13 copies the codes of each block from the pages into shared memory (bulk copies
//     of 16 tokens, which lie in one page), and the pages' scales;
//   - warps 8-11 turn them into fp16 tiles (K and V, two buffers each).  A token's row is
//     128 bytes wide in the 128-byte swizzle, in panels of 64 dims, which serves K as a
//     K-major and V as an MN-major operand.
//   - warp 12 issues the products: S = Q K^T (128 x 128 x D) and O += P V (128 x D x 128,
//     P in tensor memory).  The two halves alternate, so that one half's softmax runs
//     under the other half's products.
// What bounds it: a half's chain of scores, softmax (about 2100 cycles a block), weights and
// products (1024) and their handoffs (500), while the two halves' products are 2048.  6
// chunks of up to 2048 queries on up to 8k tokens, 32/4 heads of 128: 691 us, 1192 TFLOP/s, 0.61
// of a large bf16 product's rate; a 2123-token prefill, 64/8 heads, whose units have 1 to 17
// blocks: 98 us, 0.39.
//
// Every wait is bounded: where one runs out the call's status gets DSA_STATUS_WAIT_TIMEOUT
// and the CTA's roles stop, drain the tensor core and free its memory.  The CTAs of a
// cluster meet by its barrier, at which each of their threads comes by whatever way.
//
// Scores become u = S * (k_scale * softmax_scale * log2 e * row scaling) + (log2 v_scale - m)
// and weights 2^u (their sum: see FAR_APART), with m an integer that was the row's maximum, rounded down, when it was
// last set.  It is set anew, and O rescaled by a power of two, exactly, when a weight would
// pass 2^15, so that each fits fp16.  That is rare behind the first block.  (Sums of 64
// weights that were looked at afterwards, and the part's weights formed once more, took a
// 2123-token prefill, with its many short rows, 99.5 us against 94.9.)

#include <float.h>

#include <atomic>

#include "dsa_kv8.cuh"

namespace dsa_kv8 {

using namespace dsa;

constexpr int BLOCK = 128;       // cached tokens of a block
constexpr float MOST = 15.0f;   // largest exponent of a weight by an m that is kept
constexpr int W_DQ = 8, W_MMA = 12, W_COPY = 13, TILE_THREADS = 16 * 32;   // warps 14 and 15 only give registers
// Registers of a thread of the softmax groups and of the others: eight warps of each, which
// is what 16 warps of 128 were launched with.
constexpr int LAUNCH_REGS = 128, SOFTMAX_REGS = 152, OTHER_REGS = 104;
static_assert(SOFTMAX_REGS + OTHER_REGS == 2 * LAUNCH_REGS, "more registers than the CTA has would be waited for");
constexpr unsigned long long WAIT_LIMIT_CYCLES = 20000000000ull;   // ~10 s at 2 GHz

// barriers
enum {
  B_KFULL = 0, B_KFREE = 2, B_VFULL = 4, B_VFREE = 6,   // fp16 tiles, by buffer
  B_SFULL = 8, B_PFULL = 10, B_QFULL = 12, B_OFULL = 14,   // scores, weights, queries, result, by half
  B_RAWFULL = 16, B_RAWFREE = 18,   // codes of keys (0) and values (1)
  B_SCALES = 20, B_DRAIN = 24,
  N_BAR = 26
};
constexpr float NOTHING = -FLT_MAX;   // m of a piece in which a row saw nothing; its O is 0
constexpr int N_SCALES = 4;      // blocks whose scales are kept: see copies()

template <int D>
struct TileSmem {
  static constexpr int OPERAND = BLOCK * D * 2;   // a K, V or half-Q tile in fp16
  static constexpr int PANEL = BLOCK * 128;       // 64 dims of it
  static constexpr int RAWTILE = BLOCK * D;       // codes of a K or V block
  static constexpr int Q = 0, K = 2 * OPERAND, V = 4 * OPERAND, RAW = 6 * OPERAND, SCALES = RAW + 2 * RAWTILE;
  static constexpr int BAR = SCALES + N_SCALES * 8 * 16, MISC = BAR + 8 * N_BAR, BYTES = MISC + 32;
  static_assert(BYTES <= 227 * 1024, "shared memory of a CTA");
};
template <int D>
struct Tmem {   // columns
  static constexpr int S = 0, O = 256, COLS = 512;   // S and O of half t at S + 128 t, O + D t
};

struct Ctx {
  uint8_t* sm;
  uint32_t sb, bars;
  volatile int* misc;   // [0]: tensor memory address, [1]: abort, [2], [3]: groups of the K
                        // and V codes that have a page, [4], [5]: whether a half's unit has value scales far apart,
                        // [6]: unit whose codes are being copied, [7]: blocks copied
  uint32_t* status;
};

DSA_DEV uint32_t bar(const Ctx& c, int i) { return c.bars + 8u * (uint32_t)i; }
DSA_DEV void arrive_w(const Ctx& c, int b) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar(c, b));
}
// The waiting part of a bounded wait (in line: register counts that differ by role leave
// no room for a call).  False when the limit passes or when another thread of the CTA has
// given up.
DSA_DEV bool wait_slow(uint32_t addr, uint32_t parity, volatile int* misc, uint32_t* status) {
  const unsigned long long start = clock64();
  while (true) {
    if (mbar_wait_susp(addr, parity)) return true;
    if (misc[1]) return false;
    if (clock64() - start > WAIT_LIMIT_CYCLES) {
      atomicOr(status, DSA_STATUS_WAIT_TIMEOUT);
      misc[1] = 1;
      return false;
    }
  }
}
// The whole warp waits and agrees on the outcome.
DSA_DEV bool wait_w(const Ctx& c, int b, uint32_t parity) {
  const uint32_t addr = bar(c, b);
  const bool ok = mbar_try(addr, parity) || wait_slow(addr, parity, c.misc, c.status);
  return __all_sync(0xFFFFFFFFu, ok);
}

// Waits until unit u is being copied, or all are: for the group of a half that the unit before does
// not have.  Such units may take longer than any other wait, so this one's limit is from the last
// progress on.
DSA_DEV bool wait_unit(const Ctx& c, uint32_t u) {
  unsigned long long start = clock64();
  int blocks = c.misc[7];
  bool ok = true;
  while (ok && (int)(u - (uint32_t)c.misc[6]) > 0) {
    __nanosleep(100);
    ok = c.misc[1] == 0;
    if (c.misc[7] != blocks) {
      blocks = c.misc[7];
      start = clock64();
    }
    if (ok && clock64() - start > WAIT_LIMIT_CYCLES) {
      atomicOr(c.status, DSA_STATUS_WAIT_TIMEOUT);
      c.misc[1] = 1;
      ok = false;
    }
  }
  return __all_sync(0xFFFFFFFFu, ok);
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
DSA_DEV void commit(uint32_t bar_addr) {
  if (elect_one()) tc_commit(bar_addr);
  __syncwarp();
}

// A unit as every role sees it: the blocks of one piece of a tile, for one KV head.
struct Unit {
  Tile t;          // t.lo: of the piece
  int head, piece, pieces;
  int blocks[2];   // blocks of each half; 0 for a half without rows or without blocks in the piece
  bool rows[2];
};
// The units are in the order of the tiles, longest first; the CTAs take them forwards and
// backwards in turn, so that no CTA has the longer one of every round (forwards only, the
// first CTA of a 2123-token prefill had 40 blocks where the mean is 31).
//
// SPLIT: where there are fewer (tile, head) pairs than CTAs, a cluster of P.cluster CTAs has
// one of them, in pieces of at least two blocks, which the CTAs join in the end through
// each other's shared memory (about 3 us where a block takes 2; a join through global
// memory took 14 for 6 pieces).
template <bool SPLIT>
DSA_DEV bool unit(const Params& P, uint32_t round, int n_tiles, Unit& x) {
  // below 2^32: a unit that is not a request's last has 256 rows of q, 32 KB or more
  uint32_t u = round * gridDim.x + ((round & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
  if (SPLIT) {
    u = blockIdx.x / P.cluster;
    x.piece = blockIdx.x % P.cluster;
    if (round > 0) return false;
  }
  if (u >= (unsigned long long)n_tiles * P.h_kv) return false;
  const uint32_t i = u / (uint32_t)P.h_kv;
  x.head = (int)(u - i * P.h_kv);
  const int4* at = reinterpret_cast<const int4*>(P.tiles + i);
  // plain loads: the copying warp's bring the line to L1 for the other roles.  (Not __ldg: the
  // plan may be written while this kernel is there already.)
  const int4 a = at[0], b = at[1];
  x.t.req = a.x; x.t.row0 = a.y; x.t.q0 = a.z; x.t.rows = a.w;
  x.t.pos0 = b.x; x.t.lo = b.y; x.t.hi = b.z;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int r0 = x.t.row0 + 128 * h, r1 = min(r0 + 128, x.t.rows) - 1;
    const int hi = x.t.pos0 + r1 / P.group + 1;   // past the last token that the half sees
    x.rows[h] = r0 < x.t.rows;
    x.blocks[h] = x.rows[h] ? (hi > x.t.lo ? (hi - x.t.lo + BLOCK - 1) / BLOCK : 1) : 0;
  }
  if (!SPLIT) return true;
  const int all = max(x.blocks[0], x.blocks[1]);
  x.pieces = max(min(P.cluster, all / 2), 1);
  const int b0 = (int)((long long)all * x.piece / x.pieces), b1 = (int)((long long)all * (x.piece + 1) / x.pieces);
  x.t.lo += b0 * BLOCK;
#pragma unroll
  for (int h = 0; h < 2; ++h) x.blocks[h] = x.piece < x.pieces ? min(max(x.blocks[h] - b0, 0), b1 - b0) : 0;
  return true;
}

// ------------------------------------------------------------------------------ codes
// Lane l looks after group l of a block's eight groups of 16 tokens, each of which lies in
// one page.  A warp stops at the first use of a value that it is still loading, so a
// block's table entries are loaded two blocks ahead and its scales one block ahead.
//
// The scales of block g (counted over all units) are in slot g % 4.  They are written when
// the codes of block g - 1 have left their buffer, so the V tile of block g - 2 was written,
// so the products of block g - 4 are done: the softmax has left the slot.  The softmax reads them
// behind its wait for the scores, which come after them by way of the keys' signals; its wait for
// B_SCALES holds by itself only for a half that has had every block, since one that skipped units
// meets an older phase's parity.
template <int D, bool SPLIT>
DSA_DEV void copies(const Params& P, const Ctx& c, int n_tiles) {
  using SM = TileSmem<D>;
  constexpr uint32_t GROUP_BYTES = 16 * D;
  const int lane = threadIdx.x & 31, grp = lane & 7;
  const int page_mask = (1 << P.page_shift) - 1;
  uint32_t g = 0, u = 0;
  bool ok = true;
  Unit x;
  for (; ok && unit<SPLIT>(P, u, n_tiles, x); ++u) {
    const int blocks = max(x.blocks[0], x.blocks[1]);
    if (lane == 0) c.misc[6] = (int)u;
    const int32_t* table = P.table + x.t.req * P.table_ld;
    auto entry = [&](int i) -> int {
      const int j = x.t.lo + i * BLOCK + 16 * grp;
      return (i < blocks && j < x.t.hi) ? __ldg(table + (j >> P.page_shift)) : -1;
    };
    float ks = 1.f, vs = 1.f, least = FLT_MAX, most = 0.f;   // of this lane's groups
    auto load_scales = [&](int raw) {
      if (lane < 8 && raw >= 0 && raw < P.n_pages) {
        ks = __ldg(P.k_scale + (long long)raw * P.h_kv + x.head);
        vs = __ldg(P.v_scale + (long long)raw * P.h_kv + x.head);
      }
    };
    int raw = entry(0), raw_next = entry(1);
    load_scales(raw);
    for (int i = 0; i < blocks; ++i, ++g) {
      if (g == P.test_block && blockIdx.x == 0) {
        ok = wait_in_vain(c);
        break;
      }
      const int raw_after = entry(i + 2);
      const bool there = raw >= 0 && raw < P.n_pages;
      const uint32_t mask = __ballot_sync(0xFFFFFFFFu, there && lane < 8);
      // first row of the group in the pools
      const uint32_t row = (((uint32_t)raw * P.h_kv + x.head) << P.page_shift) +
                           ((x.t.lo + i * BLOCK + 16 * grp) & page_mask);
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        if (!(ok = wait_w(c, B_RAWFREE + kv, (g & 1) ^ 1))) break;
        if (kv == 0) {
          if (there && lane < 8) {
            least = fminf(least, bounded_scale(vs));
            most = fmaxf(most, bounded_scale(vs));
          }
          // whether the unit's value scales up to here are far apart
          const float lo = __uint_as_float(__reduce_min_sync(0xFFFFFFFFu, __float_as_uint(least)));
          const float hi = __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(most)));
          const float apart = hi > lo * FAR_APART ? 1.f : 0.f;
          if (lane < 8) {
            const float v = bounded_scale(vs);
            reinterpret_cast<float4*>(c.sm + SM::SCALES)[(g % N_SCALES) * 8 + lane] =
                there ? make_float4(ks * P.scale_log2, log2f(v), 1.0f / v, apart) : make_float4(0.f, -INFINITY, 1.f, apart);
          }
          arrive_w(c, B_SCALES + g % N_SCALES);
          load_scales(raw_next);
        }
        const uint32_t full = bar(c, B_RAWFULL + kv);
        if (lane == 0) {
          c.misc[2 + kv] = (int)mask;
          c.misc[7] = (int)g;
          asm volatile("mbarrier.arrive.expect_tx.release.cta.shared::cta.b64 _, [%0], %1;" ::"r"(full),
                       "r"((uint32_t)__popc(mask) * GROUP_BYTES)
                       : "memory");
        }
        __syncwarp();
        if (there && lane < 8) {
          const uint8_t* src = (kv == 0 ? P.k_pool : P.v_pool) + (uint64_t)row * D;
          asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                           c.sb + SM::RAW + kv * SM::RAWTILE + grp * GROUP_BYTES),
                       "l"(src), "r"(GROUP_BYTES), "r"(full)
                       : "memory");
        }
      }
      if (!ok) break;
      raw = raw_next;
      raw_next = raw_after;
    }
  }
  if (lane == 0) c.misc[6] = (int)u;
  if (!ok) {
    // gave up: wait, with a limit, for the copies in flight.  Block g's keys were issued if
    // the values' wait ran out; both buffers' last copies belong to block g or g - 1.
    const unsigned long long start = clock64();
#pragma unroll
    for (int kv = 0; kv < 2; ++kv)
      for (uint32_t b = g > 0 ? g - 1 : 0; b <= g; ++b)
        while (!mbar_wait_susp(bar(c, B_RAWFULL + kv), b & 1) && clock64() - start < WAIT_LIMIT_CYCLES / 8) {
        }
  }
}

// Block g uses buffer g % 2 of K and V.  A lane turns 16 codes into two 16-byte units of a
// swizzled row.  A quarter warp holds four chunks of an even row and the other four of the
// odd row behind it, which meet in no bank, neither here nor there.
template <int D, bool SPLIT>
DSA_DEV void dequant(const Params& P, const Ctx& c, int n_tiles) {
  using SM = TileSmem<D>;
  constexpr int CHUNKS = D / 16;            // 16-byte chunks of a row
  constexpr int ROWS = 128 / CHUNKS;        // rows of one pass of the four warps: 16 or 32
  constexpr int PASSES = BLOCK / ROWS;      // 8, or 4 for D = 64
  const int w = (threadIdx.x >> 5) - W_DQ, lane = threadIdx.x & 31;
  const int sub = w * (ROWS / 4) + (D == 128 ? (lane >> 2) & 3 : lane >> 2);   // row of a pass
  const int chunk = (lane & 3) + (D == 128 ? ((lane >> 4) ^ (sub & 1)) * 4 : 0);
  const uint32_t load_at = c.sb + SM::RAW + sub * D + 16 * chunk;
  const uint32_t store_at = c.sb + (chunk >> 2) * SM::PANEL + sub * 128;
  const uint32_t s0 = ((2 * (chunk & 3)) ^ (sub & 7)) << 4, s1 = ((2 * (chunk & 3) + 1) ^ (sub & 7)) << 4;
  uint32_t g = 0;
  Unit x;
  for (uint32_t u = 0; unit<SPLIT>(P, u, n_tiles, x); ++u) {
    const int blocks = max(x.blocks[0], x.blocks[1]);
    const int p_first = x.t.pos0 + x.t.row0 / P.group;
    const int seen_lo = P.window > 0 ? max(p_first - P.window + 1, 0) : 0;
    for (int i = 0; i < blocks; ++i, ++g) {
      const int buf = g & 1, j0 = x.t.lo + i * BLOCK;
#pragma unroll 1
      for (int kv = 0; kv < 2; ++kv) {
        if (!wait_w(c, B_RAWFULL + kv, g & 1)) return;
        const uint32_t mask = (uint32_t)c.misc[2 + kv];
        uint4 r[PASSES];
#pragma unroll
        for (int p = 0; p < PASSES; ++p)
          asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                       : "=r"(r[p].x), "=r"(r[p].y), "=r"(r[p].z), "=r"(r[p].w)
                       : "r"(load_at + kv * SM::RAWTILE + p * ROWS * D)
                       : "memory");
        if (mask != 0xFFu || (kv == 1 && (j0 < seen_lo || j0 + BLOCK > x.t.hi))) {
          // no page, or values outside what any row sees: they may be NaN codes, and
          // 0 * NaN is not 0
#pragma unroll
          for (int p = 0; p < PASSES; ++p) {
            const int row = p * ROWS + sub, j = j0 + row;
            if (!((mask >> (row >> 4)) & 1u) || (kv == 1 && (j < seen_lo || j >= x.t.hi))) r[p] = make_uint4(0u, 0u, 0u, 0u);
          }
        }
        arrive_w(c, B_RAWFREE + kv);   // the codes are in registers
        if (!wait_w(c, (kv ? B_VFREE : B_KFREE) + buf, ((g >> 1) & 1) ^ 1)) return;
        const uint32_t to = store_at + (kv ? SM::V : SM::K) + buf * SM::OPERAND;
#pragma unroll
        for (int p = 0; p < PASSES; ++p) {
          uint32_t h[8];
          codes16_to_f16(r[p], h);
          sts128(to + p * ROWS * 128 + s0, make_uint4(h[0], h[1], h[2], h[3]));
          sts128(to + p * ROWS * 128 + s1, make_uint4(h[4], h[5], h[6], h[7]));
        }
        fence_async_smem();
        arrive_w(c, (kv ? B_VFULL : B_KFULL) + buf);
      }
    }
  }
}

DSA_DEV uint32_t ld_shared(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

// ------------------------------------------------------------------------------ products
// The whole warp runs this role and one elected lane issues each product: with
// warp-uniform control flow the descriptors stay in uniform registers.
template <int D, bool SPLIT>
DSA_DEV void products(const Params& P, const Ctx& c, uint32_t tmem, int n_tiles) {
  using SM = TileSmem<D>;
  using TM = Tmem<D>;
  constexpr uint32_t ID_QK = idesc_f16(128, BLOCK, 0, 0);
  constexpr uint32_t ID_PV = idesc_f16(128, D, 0, 1);
  const uint64_t d_q = sdesc(c.sb + SM::Q, 16, 1024);
  const uint64_t d_k = sdesc(c.sb + SM::K, 16, 1024);
  const uint64_t d_v = sdesc(c.sb + SM::V, SM::PANEL, 1024);
  uint32_t g = 0;                 // blocks
  uint32_t np[2] = {0, 0};        // blocks of each half
  uint32_t nq[2] = {0, 0};        // units of each half
  Unit x;
  for (uint32_t u = 0; unit<SPLIT>(P, u, n_tiles, x); ++u) {
    const int blocks = max(x.blocks[0], x.blocks[1]);
    for (int i = 0; i <= blocks; ++i) {
      const int kb = (g + i) & 1, vb = kb ^ 1;
      // the values of a block are written before the next one's keys
      if (i < blocks && !wait_w(c, B_KFULL + kb, ((g + i) >> 1) & 1)) return;
      if (i > 0 && i == blocks && !wait_w(c, B_VFULL + vb, ((g + i - 1) >> 1) & 1)) return;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const bool pv = i > 0 && i - 1 < x.blocks[h], qk = i < x.blocks[h];
        if (pv) {
          if (!wait_w(c, B_PFULL + h, np[h] & 1)) return;
          ++np[h];
        } else if (qk) {
          if (!wait_w(c, B_QFULL + h, nq[h] & 1)) return;
          ++nq[h];
        }
        tc_fence_after();
        if (elect_one()) {
          if (pv) {
#pragma unroll
            for (int k = 0; k < BLOCK / 16; ++k)
              mma_ts(tmem + TM::O + D * h, tmem + TM::S + 128 * h + 8 * k,
                     d_v + ((uint32_t)(vb * SM::OPERAND + k * 2048) >> 4), ID_PV, (i > 1 || k > 0) ? 1u : 0u);
            if (!qk) {
              // from the half's last block, whose scales stay until these products are done.  (Read by the
              // softmax with every block it took 0.5 % longer; a branch in its loop, 5 %.)
              const uint32_t at = c.sb + SM::SCALES + (g + i - 1) % N_SCALES * 128 + 12;
              c.misc[4 + h] = ld_shared(at) != 0;
              mbar_arrive(bar(c, B_OFULL + h));
              tc_commit(bar(c, B_OFULL + h));
            }
          }
          if (qk) {
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
              const uint32_t off = (k >> 2) * SM::PANEL + (k & 3) * 32;
              mma_ss(tmem + TM::S + 128 * h, d_q + ((h * SM::OPERAND + off) >> 4), d_k + ((kb * SM::OPERAND + off) >> 4),
                     ID_QK, k ? 1u : 0u);
            }
            tc_commit(bar(c, B_SFULL + h));
          }
          if (h == 1) {
            if (i < blocks) tc_commit(bar(c, B_KFREE + kb));
            if (i > 0) tc_commit(bar(c, B_VFREE + vb));
          }
        }
        __syncwarp();
      }
    }
    g += blocks;
  }
}

// ------------------------------------------------------------------------------ softmax
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

DSA_DEV const uint16_t* shfl_ptr(const uint16_t* p, int from) {
  return reinterpret_cast<const uint16_t*>(__shfl_sync(0xFFFFFFFFu, reinterpret_cast<unsigned long long>(p), from));
}

// Whether a row sees a cached token of a unit's blocks.
DSA_DEV bool sees_any(const Params& P, const Unit& x, int blocks, int pos) {
  const int32_t* table = P.table + x.t.req * P.table_ld;
  const int end = min(min(x.t.lo + blocks * BLOCK, x.t.hi), pos + 1);
  const int first = P.window > 0 ? max(x.t.lo, pos - P.window + 1) : x.t.lo;
  for (int j = first & ~(STEP - 1); j < end; j += STEP) {   // a step lies in one page
    const int page = __ldg(table + (j >> P.page_shift));
    if (page >= 0 && page < P.n_pages) return true;
  }
  return false;
}

// Scales the warp's 32 rows of queries to fp16 and writes them into a half's tile.  `mine`
// is this lane's row, null for one that is not there, and `row0` the warp's first row of
// the tile.  Returns what undoes the scaling of this lane's row.  Lanes side by side read
// neighbours of a row: a lane for a row touches 32 lines with every load, which took a
// 2123-token prefill 109 us in place of 104.
//
// A query that is not finite makes its row NaN, also by way of missing pages (0 * NaN); where the
// row sees nothing it has to be 0, and the query is taken as 0.
template <int D, bool FP16>
DSA_DEV float queries(const Params& P, const Unit& x, int blocks, int pos, const uint16_t* mine, uint32_t tile, int row0) {
  constexpr int LANES = D / 8, AT_ONCE = 32 / LANES;   // lanes of a row, rows of a load; LANES loads
  const int lane = threadIdx.x & 31, sub = lane / LANES, chunk = lane % LANES;
  uint4 v[LANES];
#pragma unroll
  for (int t = 0; t < LANES; ++t) {
    const uint16_t* src = shfl_ptr(mine, AT_ONCE * t + sub);
    v[t] = src ? ldg_nc(src + 8 * chunk) : make_uint4(0u, 0u, 0u, 0u);
  }
  // largest magnitudes, as 16-bit patterns in pairs: lane l ends with those of load l % LANES
  uint32_t mx[LANES];
#pragma unroll
  for (int t = 0; t < LANES; ++t)
    mx[t] = __vmaxu2(__vmaxu2(v[t].x & 0x7FFF7FFFu, v[t].y & 0x7FFF7FFFu), __vmaxu2(v[t].z & 0x7FFF7FFFu, v[t].w & 0x7FFF7FFFu));
#pragma unroll
  for (int n = LANES / 2; n >= 1; n >>= 1)
#pragma unroll
    for (int j = 0; j < n; ++j) {
      const bool high = lane & n;
      mx[j] = __vmaxu2(high ? mx[j + n] : mx[j], __shfl_xor_sync(0xFFFFFFFFu, high ? mx[j] : mx[j + n], n));
    }
  float back;
  const uint32_t largest = max(mx[0] >> 16, mx[0] & 0xFFFFu);
  const int holder = lane / AT_ONCE + lane % AT_ONCE * LANES;   // of what belongs to this lane's row
  const bool finite = largest < (FP16 ? 0x7C00u : 0x7F80u);
  if (!__all_sync(0xFFFFFFFFu, finite)) {
    const bool none = !__shfl_sync(0xFFFFFFFFu, finite, holder) && !sees_any(P, x, blocks, pos);
#pragma unroll
    for (int t = 0; t < LANES; ++t)
      if (__shfl_sync(0xFFFFFFFFu, none, AT_ONCE * t + sub)) v[t] = make_uint4(0u, 0u, 0u, 0u);
  }
  const float down = row_scaling(unpack(largest, FP16).x, back);
  const uint32_t at = tile + (chunk >> 3) * (BLOCK * 128) + (row0 + sub) * 128;
#pragma unroll
  for (int t = 0; t < LANES; ++t) {
    const float f = __shfl_sync(0xFFFFFFFFu, down, sub * LANES + t);
    uint32_t p[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 y = unpack(word(v[t], e), FP16);
      p[e] = pack_f16x2(y.x * f, y.y * f);
    }
    sts128(at + AT_ONCE * t * 128 + (((chunk ^ (AT_ONCE * t + sub)) & 7) << 4), make_uint4(p[0], p[1], p[2], p[3]));
  }
  return __shfl_sync(0xFFFFFFFFu, back, holder);
}

DSA_DEV void cluster_meet() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
DSA_DEV uint32_t at_rank(uint32_t addr, int rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
  return a;
}
DSA_DEV float ld_cluster(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
DSA_DEV float4 ld_cluster4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
  return v;
}

// The sum of 2^(score - m) over what a row sees of a unit's blocks, each score formed anew from the
// row's queries in shared memory and the codes: for a unit whose value scales are far apart.
template <int D>
DSA_DEV float plain_sum(const Params& P, const Unit& x, const uint8_t* tile, int row_in, int blocks, int pos, float row_scale,
                        float m) {
  const int32_t* table = P.table + x.t.req * P.table_ld;
  const int end = min(min(x.t.lo + blocks * BLOCK, x.t.hi), pos + 1);
  float sum = 0.f;
  for (int j = P.window > 0 ? max(x.t.lo, pos - P.window + 1) : x.t.lo; j < end; ++j) {
    const int page = __ldg(table + (j >> P.page_shift));
    if (page < 0 || page >= P.n_pages) continue;
    const uint32_t unit = (uint32_t)page * P.h_kv + x.head;
    const uint32_t row = (unit << P.page_shift) + (j & ((1 << P.page_shift) - 1));
    const uint8_t* k = P.k_pool + (uint64_t)row * D;
    float dot = 0.f;
#pragma unroll 1
    for (int c8 = 0; c8 < D / 8; ++c8) {
      const uint2 codes = ldg_nc_v2(k + 8 * c8);
      const uint4 q = *reinterpret_cast<const uint4*>(tile + (c8 >> 3) * (BLOCK * 128) + row_in * 128 + (((c8 ^ row_in) & 7) << 4));
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t h2 = e4m3x2_to_f16x2(((e < 2 ? codes.x : codes.y) >> (16 * (e & 1))) & 0xFFFFu);
        const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&h2)), b = unpack(word(q, e), 1);
        dot = fmaf(a.x, b.x, fmaf(a.y, b.y, dot));
      }
    }
    sum += ex2(fmaf(dot, __ldg(P.k_scale + unit) * P.scale_log2 * row_scale, -m));
  }
  return sum;
}

// Returns whether the CTA's cluster has met (SPLIT).
template <int D, bool SPLIT>
DSA_DEV bool softmax(const Params& P, const Ctx& c, uint32_t tmem, int n_tiles, int h) {
  using SM = TileSmem<D>;
  using TM = Tmem<D>;
  const int row_in = threadIdx.x & 127;
  const uint32_t lanes = (uint32_t)((threadIdx.x >> 5) & 3) << 21;   // the warp's 32 lanes of tensor memory
  const uint32_t ts = tmem + lanes + TM::S + 128 * h, to = tmem + lanes + TM::O + D * h;
  uint32_t g = 0, ns = 0, no = 0;
  bool met = false;
  Unit x;
  for (uint32_t u = 0; unit<SPLIT>(P, u, n_tiles, x); ++u) {
    const int blocks = max(x.blocks[0], x.blocks[1]), mine = h == 0 ? x.blocks[0] : x.blocks[1];
    if (!(h == 0 ? x.rows[0] : x.rows[1]) || (SPLIT && x.piece >= x.pieces)) {
      g += blocks;
      if (!SPLIT && !wait_unit(c, u + 1)) return met;
      continue;
    }
    const int first = x.t.row0 + 128 * h, row = first + row_in;
    const bool live = row < x.t.rows;
    const int qi = min(row, x.t.rows - 1) / P.group;
    const int pos = x.t.pos0 + qi;
    const int pos_min = x.t.pos0 + first / P.group, pos_max = x.t.pos0 + min(first + 127, x.t.rows - 1) / P.group;
    const int head = x.head * P.group + row - qi * P.group;
    // ---- the query row (its buffer was last read for this half's last scores)
    float row_scale = 1.0f;
    if (!SPLIT || mine > 0) {
      const uint16_t* src = live ? P.q + (x.t.q0 + qi) * P.q_ld + head * P.q_hd : nullptr;
      const uint32_t tile = c.sb + SM::Q + h * SM::OPERAND;
      row_scale = P.fp16 ? queries<D, true>(P, x, mine, pos, src, tile, row_in & ~31)
                         : queries<D, false>(P, x, mine, pos, src, tile, row_in & ~31);
      fence_async_smem();
      tc_fence_before();   // this half's O was read before
      arrive_w(c, B_QFULL + h);
    }
    float m = 0.f, l = 0.f;
    bool fresh = true;   // m is not set: every score so far was masked
    for (int i = 0; i < mine; ++i) {
      const uint32_t gi = g + i;
      if (!wait_w(c, B_SCALES + gi % N_SCALES, (gi / N_SCALES) & 1)) return met;
      const float4* sc = reinterpret_cast<const float4*>(c.sm + SM::SCALES) + (gi % N_SCALES) * 8;
      const int base = x.t.lo + i * BLOCK;
      if (!wait_w(c, B_SFULL + h, ns & 1)) return met;
      ++ns;
      tc_fence_after();
#pragma unroll 1
      for (int s = 0; s < 2; ++s) {   // 64 tokens at a time: two copies of this code cost more than they gain
        uint32_t x2[64];
        tmem_ld32(ts + 64 * s, *reinterpret_cast<uint32_t(*)[32]>(x2));
        tmem_ld32(ts + 64 * s + 32, *reinterpret_cast<uint32_t(*)[32]>(x2 + 32));
        float2 mul_add[4];
        float vinv[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float4 f = sc[4 * s + q];
          mul_add[q] = make_float2(f.x * row_scale, f.y - m);
          vinv[q] = f.z;
        }
        tc_wait_ld();
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const uint64_t mul = pair(mul_add[q].x, mul_add[q].x), add = pair(mul_add[q].y, mul_add[q].y);
#pragma unroll
          for (int e = 0; e < 16; e += 2) fma2(x2[16 * q + e], x2[16 * q + e + 1], mul, add);
        }
        const int j0 = base + 64 * s;
        if (j0 + 63 > pos_min || (P.window > 0 && j0 <= pos_max - P.window)) {
          const int last = pos - j0, before = P.window > 0 ? last - P.window : -1;
#pragma unroll
          for (int e = 0; e < 64; ++e)
            if (e > last || e <= before) x2[e] = 0xFF800000u;   // -inf
        }
        float t4[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          t4[q] = fmaxf(__uint_as_float(x2[q]), __uint_as_float(x2[q + 4]));
#pragma unroll
          for (int e = 8; e < 64; e += 8) t4[q] = max3(t4[q], __uint_as_float(x2[e + q]), __uint_as_float(x2[e + 4 + q]));
        }
        const float top = fmaxf(max3(t4[0], t4[1], t4[2]), t4[3]);
        if (__any_sync(0xFFFFFFFFu, fresh || top > MOST)) {
          // what this thread stored last (O, or the weights of the block's first part) is read
          // again below, and only this wait puts a tensor memory load behind a store
          tc_wait_st();
          const bool up = top > (fresh ? -INFINITY : LAG);
          // The largest weight is in [1, 2), and it is by delta that weights and sums are rescaled: from 2^23 on
          // m + delta is rounded, and weights by m's rounded step (2^5 and more for scores from 2^28 on) would
          // pass fp16's range.
          const float delta = up ? floorf(top) : 0.f;
          const float to_m = m + delta, f = (up && !fresh) ? ex2(-delta) : 1.0f;
          if (up) fresh = false;
          m = to_m;
          l *= f;
#pragma unroll
          for (int e = 0; e < 64; ++e) x2[e] = __float_as_uint(__uint_as_float(x2[e]) - delta);
          if (__any_sync(0xFFFFFFFFu, f != 1.0f)) {
            if (i > 0) {
              // the product of the block before is done: these scores were issued after it
#pragma unroll 1
              for (int k = 0; k < D; k += 32) {
                uint32_t o[32];
                tmem_ld32(to + k, o);
                tc_wait_ld();
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                tmem_st32(to + k, o);
              }
            }
            if (s == 1) {   // the weights of the block's first part; in fp32, where f has all its range
#pragma unroll 1
              for (int k = 0; k < 32; k += 16) {
                uint32_t o[16];
                tmem_ld16(ts + k, o);
                tc_wait_ld();
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                  const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&o[e]));
                  o[e] = pack_f16x2(y.x * f, y.y * f);
                }
                tmem_st16(ts + k, o);
              }
            }
          }
        }
        uint32_t p[32];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          float s0 = 0.f, s1 = 0.f;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float w0 = ex2(__uint_as_float(x2[16 * q + 2 * e])), w1 = ex2(__uint_as_float(x2[16 * q + 2 * e + 1]));
            add2(s0, s1, w0, w1);
            p[8 * q + e] = pack_f16x2(w0, w1);
          }
          l = fmaf(s0 + s1, vinv[q], l);
        }
        tmem_st32(ts + 32 * s, p);
      }
      tc_wait_st();
      tc_fence_before();
      arrive_w(c, B_PFULL + h);
    }
    // ---- result
    if (!SPLIT || mine > 0) {
      if (!wait_w(c, B_OFULL + h, no & 1)) return met;
      ++no;
      tc_fence_after();
      if (c.misc[4 + h])
        l = live ? plain_sum<D>(P, x, c.sm + SM::Q + h * SM::OPERAND, row_in, mine, pos, row_scale, m) : 0.f;
    }
    uint16_t* dst = P.out + (x.t.q0 + qi) * P.out_ld + head * P.out_hd;
    auto write = [&](int k, const float* o, float inv) {   // 8 dims
      if (!live) return;
      uint4 v;
      v.x = pack(o[0] * inv, o[1] * inv, P.fp16);
      v.y = pack(o[2] * inv, o[3] * inv, P.fp16);
      v.z = pack(o[4] * inv, o[5] * inv, P.fp16);
      v.w = pack(o[6] * inv, o[7] * inv, P.fp16);
      *reinterpret_cast<uint4*>(dst + k) = v;
    };
    auto inverse = [](float sum) { return sum > 0.f ? 1.0f / sum : (sum == 0.f ? 0.f : sum); };   // a NaN sum stays one
    if (!SPLIT || x.pieces == 1) {
      const float inv = inverse(l);
#pragma unroll 1
      for (int k = 0; k < D; k += 32) {
        uint32_t o[32];
        tmem_ld32(to + k, o);
        tc_wait_ld();
#pragma unroll
        for (int e = 0; e < 32; e += 8) write(k + e, reinterpret_cast<const float*>(o) + e, inv);
      }
    } else {
      // One of several pieces.  O of both halves goes over the K and V tiles, whose products
      // are done, as [D / 4][128 rows][4]; m and l over the codes.
      const int other = h == 0 ? x.blocks[1] : x.blocks[0];
      if (other > 0 && !wait_w(c, B_OFULL + 1 - h, 0)) return met;
      const uint32_t s_o = c.sb + SM::K + 2 * SM::OPERAND * h, s_ml = c.sb + SM::RAW + 1024 * h;
#pragma unroll 1
      for (int k = 0; k < D; k += 32) {
        uint32_t o[32];
        if (mine > 0) {
          tmem_ld32(to + k, o);
          tc_wait_ld();
        }
#pragma unroll
        for (int e = 0; e < 8; ++e)
          sts128(s_o + ((k / 4 + e) * 128 + row_in) * 16,
                 mine > 0 ? make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]) : make_uint4(0u, 0u, 0u, 0u));
      }
      float* ml = reinterpret_cast<float*>(c.sm + SM::RAW + 1024 * h);
      ml[row_in] = fresh ? NOTHING : m;
      ml[128 + row_in] = l;
      cluster_meet();
      met = true;
      // this CTA joins 8-dim chunks [c0, c1) of every row, in the order of the pieces
      m = NOTHING;
      for (int p = 0; p < x.pieces; ++p) m = fmaxf(m, ld_cluster(at_rank(s_ml, p) + 4 * row_in));
      l = 0.f;
      for (int p = 0; p < x.pieces; ++p) {
        const uint32_t from = at_rank(s_ml, p) + 4 * row_in;
        l += scaled(ld_cluster(from + 512), ld_cluster(from) - m);
      }
      const float inv = inverse(l);
      const int c0 = D / 8 * x.piece / x.pieces, c1 = D / 8 * (x.piece + 1) / x.pieces;
      for (int k = c0; k < c1; ++k) {
        float o[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = 0.f;
#pragma unroll 4
        for (int p = 0; p < x.pieces; ++p) {
          const float f = ex2(ld_cluster(at_rank(s_ml, p) + 4 * row_in) - m);
          const uint32_t from = at_rank(s_o, p) + (2 * k * 128 + row_in) * 16;
          const float4 a = ld_cluster4(from), b = ld_cluster4(from + 128 * 16);
          o[0] = fmaf(a.x, f, o[0]); o[1] = fmaf(a.y, f, o[1]); o[2] = fmaf(a.z, f, o[2]); o[3] = fmaf(a.w, f, o[3]);
          o[4] = fmaf(b.x, f, o[4]); o[5] = fmaf(b.y, f, o[5]); o[6] = fmaf(b.z, f, o[6]); o[7] = fmaf(b.w, f, o[7]);
        }
        write(8 * k, o, inv);
      }
    }
    if (live && P.lse && (!SPLIT || x.piece == 0))
      P.lse[(long long)(x.t.q0 + qi) * P.h_q + head] = l == 0.f ? -INFINITY : 0.6931471805599453f * (m + log2f(l));
    g += blocks;
  }
  return met;
}

template <int D, bool SPLIT>
__global__ void __launch_bounds__(TILE_THREADS, 1) tiles_kernel(const __grid_constant__ Params P) {
  extern __shared__ __align__(1024) uint8_t smem[];
  using SM = TileSmem<D>;
  Ctx c;
  c.sm = smem;
  c.sb = smem_u32(smem);
  c.bars = c.sb + SM::BAR;
  c.misc = reinterpret_cast<volatile int*>(smem + SM::MISC);
  c.status = &P.header->status;
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(c, B_KFULL + i), 4);
      mbar_init(bar(c, B_KFREE + i), 1);
      mbar_init(bar(c, B_VFULL + i), 4);
      mbar_init(bar(c, B_VFREE + i), 1);
      mbar_init(bar(c, B_SFULL + i), 1);
      mbar_init(bar(c, B_PFULL + i), 4);
      mbar_init(bar(c, B_QFULL + i), 4);
      mbar_init(bar(c, B_OFULL + i), 2);
      mbar_init(bar(c, B_RAWFULL + i), 1);
      mbar_init(bar(c, B_RAWFREE + i), 4);
    }
    for (int i = 0; i < N_SCALES; ++i) mbar_init(bar(c, B_SCALES + i), 1);
    mbar_init(bar(c, B_DRAIN), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    c.misc[1] = c.misc[6] = c.misc[7] = 0;
  }
  if (warp == W_MMA) tmem_alloc(c.sb + SM::MISC, Tmem<D>::COLS);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = (uint32_t)c.misc[0];
  // launched as a programmatic dependent of rows_kernel, which waited for the plan
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int n_tiles = P.header->n_tiles;
  bool met = false;
  if (warp < W_DQ) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(SOFTMAX_REGS));
    met = softmax<D, SPLIT>(P, c, tmem, n_tiles, warp >> 2);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(OTHER_REGS));
    if (warp < W_MMA) dequant<D, SPLIT>(P, c, n_tiles);
    else if (warp == W_MMA) products<D, SPLIT>(P, c, tmem, n_tiles);
    else if (warp == W_COPY) copies<D, SPLIT>(P, c, n_tiles);
  }
  if (SPLIT) {   // every thread twice: the pieces are there; and they have been read
    if (!met) cluster_meet();
    cluster_meet();
  }
  if (warp == W_MMA) commit(bar(c, B_DRAIN));
  tc_fence_before();
  __syncthreads();
  if (warp == W_MMA && (threadIdx.x & 31) == 0) {
    // every product has completed before tensor memory is released
    const unsigned long long start = clock64();
    while (!mbar_wait_susp(bar(c, B_DRAIN), 0) && clock64() - start < WAIT_LIMIT_CYCLES) {
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == W_MMA) {
    tc_fence_after();
    tmem_dealloc(tmem, Tmem<D>::COLS);
  }
}

template <int D, bool SPLIT>
static int configure(const Params& P, cudaLaunchConfig_t& cfg, cudaLaunchAttribute (&attr)[2], cudaStream_t st) {
  constexpr int smem = TileSmem<D>::BYTES;
  // the kernel's groups trade the registers that its launch gave them
  cudaFuncAttributes a;
  if (cudaFuncGetAttributes(&a, tiles_kernel<D, SPLIT>) != cudaSuccess || a.numRegs != LAUNCH_REGS) return DSA_ERR_CUDA;
  if (cudaFuncSetAttribute(tiles_kernel<D, SPLIT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
    return DSA_ERR_CUDA;
  if (SPLIT && cudaFuncSetAttribute(tiles_kernel<D, SPLIT>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess)
    return DSA_ERR_CUDA;
  cfg = {};
  cfg.gridDim = dim3((unsigned)P.n_ctas);
  cfg.blockDim = dim3(TILE_THREADS);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)max(P.cluster, 1);
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = SPLIT ? 2 : 1;
  return DSA_OK;
}

template <int D, bool SPLIT>
static int launch_one(const Params& P, cudaStream_t st) {
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[2];
  const int rc = configure<D, SPLIT>(P, cfg, attr, st);
  if (rc != DSA_OK) return rc;
  return cudaLaunchKernelEx(&cfg, tiles_kernel<D, SPLIT>, P) == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}

// How many clusters of a size the current device holds at a time: a property of the device,
// asked for once.
template <int D>
static int resident_clusters(int size) {
  constexpr int DEVICES = 64;
  static std::atomic<int> known[DEVICES][MAX_CLUSTER + 1];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (dev < DEVICES && known[dev][size].load(std::memory_order_relaxed) > 0) return known[dev][size].load(std::memory_order_relaxed) - 1;
  Params P = {};
  P.n_ctas = P.cluster = size;
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[2];
  int n = 0;
  if (configure<D, true>(P, cfg, attr, nullptr) != DSA_OK) return 0;
  cfg.attrs = attr + 1;   // the cluster's
  cfg.numAttrs = 1;
  if (cudaOccupancyMaxActiveClusters(&n, tiles_kernel<D, true>, &cfg) != cudaSuccess) {
    cudaGetLastError();   // a size that this device cannot hold
    n = 0;
  }
  if (dev < DEVICES) known[dev][size].store(n + 1, std::memory_order_relaxed);
  return n;
}

int cluster_size(int d, long long units, int blocks) {
  if (blocks < 4) return 0;   // no two pieces of two blocks
  for (const int size : {12, 10, 8, 6, 4, 2})
    if ((size <= blocks / 2 || size == 2) && units <= (d == 128 ? resident_clusters<128>(size) : resident_clusters<64>(size)))
      return size;
  return 0;
}

// The kernel that splits a tile's blocks is a copy of its own: with the joining in it, the
// other one's loops took a tenth longer.
int launch_tiles(int d, const Params& P, cudaStream_t st) {
  if (P.cluster) return d == 128 ? launch_one<128, true>(P, st) : launch_one<64, true>(P, st);
  return d == 128 ? launch_one<128, false>(P, st) : launch_one<64, false>(P, st);
}

}  // namespace dsa_kv8
