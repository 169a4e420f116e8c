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

constexpr unsigned PIECE_BLOCKS = 2;   // blocks that take a CTA as long as a piece's beginning and end

// Blocks of each CTA where all get as many, and CTAs of a unit of `len` of all `total` blocks where each unit
// has CTAs of its own.  (len * n_ctas is below 2^32: see prefix_layout().)
DSA_HD unsigned equal_blocks(unsigned total, unsigned n_ctas) {
  const unsigned each = (total + n_ctas - 1) / n_ctas;
  return each > 2 ? each : 2;
}
DSA_HD unsigned own_ctas(unsigned len, unsigned total, unsigned n_ctas) {
  const unsigned part = len * n_ctas / total, most = part < len / 2 ? part : len / 2;
  return most > 1 ? most : 1;
}
// Whether each unit gets CTAs of its own, which leaves each CTA one piece to begin and to end: where these are
// as many as there are (own_ctas() gives a short unit one, whatever its part of the blocks, so that the sum may
// pass them) and none gets PIECE_BLOCKS more than by equal shares.
DSA_HD bool own_pieces(unsigned long long all_ctas, unsigned n_ctas, unsigned longest, unsigned each) {
  return all_ctas <= n_ctas && longest <= each + PIECE_BLOCKS;
}

struct Cuts {
  const unsigned* before;   // [n_tiles + 1] blocks of a head in front of each tile
  const unsigned* front;    // [n_tiles + 1] CTAs in front of each tile's
  const unsigned* ctas;     // [n_tiles] of a unit of each tile
  unsigned n_tiles, h_kv, each;
  bool own;                 // own_pieces()

  // cut b, and the unit that is there (n_tiles * h_kv: none)
  DSA_HD unsigned cut(unsigned b, unsigned& unit) const {
    const unsigned* starts = own ? front : before;
    const unsigned scale = own ? 1 : h_kv, at = own ? b : b * each;
    unit = n_tiles * h_kv;
    if (at >= starts[n_tiles] * scale) return before[n_tiles] * h_kv;
    unsigned lo = 0, hi = n_tiles;   // the tile with starts[lo] * scale <= at < starts[lo + 1] * scale
    while (hi - lo > 1) {
      const unsigned mid = (lo + hi) >> 1;
      if (starts[mid] * scale <= at) lo = mid; else hi = mid;
    }
    const unsigned rest = at - starts[lo] * scale, len = before[lo + 1] - before[lo], k = ctas[lo];
    const unsigned head = rest / (own ? k : len);
    unit = lo * h_kv + head;
    return own ? before[lo] * h_kv + head * len + len * (rest - head * k) / k : at;
  }
  // the first and the last CTA of a unit
  DSA_HD void ctas_of(unsigned unit, int& first, int& last) const {
    const unsigned i = unit / h_kv, head = unit - i * h_kv, len = before[i + 1] - before[i];
    const unsigned from = before[i] * h_kv + head * len, b = front[i] + head * ctas[i];
    first = (int)(own ? b : from / each);
    last = (int)(own ? b + ctas[i] - 1 : (from + len - 1) / each);
  }
};

}  // namespace dsa_kv8
