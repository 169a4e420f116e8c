// How the blocks of few tiles are shared out to the CTAs of the tiles' kernel (dsa_kv8_prefix.cu), in integers
// alone: the plan kernel computes with these, and a host can.
//
// A unit is a tile and a KV head.  All units' blocks lie in a row, those of a tile's first head in front of
// those of its second.  CTA b takes the blocks from cut b up to cut b + 1.
#pragma once

#ifdef __CUDACC__
#define DSA_HD __host__ __device__ __forceinline__
#else
#define DSA_HD inline
#endif

namespace dsa_kv8 {

constexpr unsigned PIECE_BLOCKS = 2;   // how many blocks more than others a CTA may get for the sake of a single piece
// What a unit costs a CTA beside its blocks, in blocks, where shares are equal: the units of one block, which lie side
// by side, would else come to a few CTAs.  us, with 0, 2, 4, 6 and 8, 64/8 heads of 128: 4 requests of 128 queries behind
// 16k tokens 978, 476, 314, 271 and 279; 16 of 16 queries 538, 216, 155, 159 and 163; 12 of 6 queries behind 8k 104, 63,
// 61, 65 and 67; one query each of 8 requests behind 16k and of twice 8 behind 256 tokens 71, 56, 56, 56 and 58.
constexpr unsigned UNIT_BLOCKS = 4;

// Blocks of each CTA where all get as many, and the same with what their units cost
DSA_HD unsigned equal_blocks(unsigned total, unsigned n_ctas) {
  const unsigned each = (total + n_ctas - 1) / n_ctas;
  return each > 2 ? each : 2;
}
DSA_HD unsigned equal_costs(unsigned total, unsigned units, unsigned n_ctas) {
  const unsigned each = (total + units * UNIT_BLOCKS + n_ctas - 1) / n_ctas;
  return each > UNIT_BLOCKS + 2 ? each : UNIT_BLOCKS + 2;
}
// CTAs of a unit of `len` of all `total` blocks where each unit has CTAs of its own.  (len * n_ctas is below
// 2^32: see prefix_layout().)
DSA_HD unsigned own_ctas(unsigned len, unsigned total, unsigned n_ctas) {
  const unsigned part = len * n_ctas / total, most = part < len / 2 ? part : len / 2;
  return most > 1 ? most : 1;
}
// Whether each unit gets CTAs of its own, which leaves each CTA one piece to begin and to end: where these are
// as many as there are (own_ctas() gives a short unit one, whatever its part of the blocks, so that the sum may
// pass them) and none gets more than PIECE_BLOCKS above `each`, equal_blocks().
DSA_HD bool own_pieces(unsigned long long all_ctas, unsigned n_ctas, unsigned longest, unsigned each) {
  return all_ctas <= n_ctas && longest <= each + PIECE_BLOCKS;
}

struct Cuts {
  const unsigned* before;   // [n_tiles + 1] blocks of a head in front of each tile
  const unsigned* front;    // [n_tiles + 1] CTAs in front of each tile's, where units have their own
  const unsigned* ctas;     // [n_tiles] of a unit of each tile
  unsigned n_tiles, h_kv;
  unsigned each;            // equal_costs()
  bool own;                 // own_pieces()

  // Where tile i's CTAs begin, or its costs: block j of a unit whose costs begin at c is at c + UNIT_BLOCKS + j
  // there, and CTA b has the blocks at b * each and behind.
  DSA_HD unsigned start(unsigned i) const { return own ? front[i] : (before[i] + i * UNIT_BLOCKS) * h_kv; }
  // cut b, and the unit that is there (n_tiles * h_kv: none)
  DSA_HD unsigned cut(unsigned b, unsigned& unit) const {
    const unsigned at = own ? b : b * each;
    unit = n_tiles * h_kv;
    if (at >= start(n_tiles)) return before[n_tiles] * h_kv;
    unsigned lo = 0, hi = n_tiles;   // the tile with start(lo) <= at < start(lo + 1)
    while (hi - lo > 1) {
      const unsigned mid = (lo + hi) >> 1;
      if (start(mid) <= at) lo = mid; else hi = mid;
    }
    const unsigned len = before[lo + 1] - before[lo], size = own ? ctas[lo] : len + UNIT_BLOCKS;
    const unsigned head = (at - start(lo)) / size, rest = at - start(lo) - head * size;
    unit = lo * h_kv + head;
    return before[lo] * h_kv + head * len + (own ? len * rest / size : rest > UNIT_BLOCKS ? rest - UNIT_BLOCKS : 0);
  }
  // the first and the last CTA of a unit
  DSA_HD void ctas_of(unsigned unit, int& first, int& last) const {
    const unsigned i = unit / h_kv, head = unit - i * h_kv, len = before[i + 1] - before[i];
    const unsigned at = start(i) + head * (own ? ctas[i] : len + UNIT_BLOCKS);
    first = (int)(own ? at : (at + UNIT_BLOCKS) / each);
    last = (int)(own ? at + ctas[i] - 1 : (at + UNIT_BLOCKS + len - 1) / each);
  }
};

}  // namespace dsa_kv8
