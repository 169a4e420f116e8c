"""How the tiles of the attention for requests that share prefixes are cut for the CTAs (no GPU): the plan kernel's own integers
(csrc/dsa_kv8_cuts.h), compiled for the host.  Every block of every unit has to belong to one CTA, and the CTAs that a unit is said
to have, whose pieces are joined, have to be those."""

import ctypes
import os
import random
import subprocess

import pytest

from top_sparse_mla_gb300.build import PKG_DIR

SOURCE = r"""
#include "dsa_kv8_cuts.h"
#include <algorithm>
#include <vector>
// As the plan kernel does.  cuts, units [n_ctas + 1]; by [2 n_tiles h_kv].  Returns whether units have CTAs of their own.
extern "C" int plan(const unsigned* len, unsigned n_tiles, unsigned h_kv, unsigned n_ctas, unsigned* cuts, unsigned* units, int* by) {
  using namespace dsa_kv8;
  std::vector<unsigned> before(n_tiles + 1), front(n_tiles + 1), ctas(n_tiles);
  for (unsigned i = 0; i < n_tiles; ++i) before[i + 1] = before[i] + len[i];
  const unsigned total = before[n_tiles] * h_kv;
  unsigned longest = 0;
  for (unsigned i = 0; i < n_tiles; ++i) {
    ctas[i] = own_ctas(len[i], total, n_ctas);
    front[i + 1] = front[i] + ctas[i] * h_kv;
    longest = std::max(longest, (len[i] + ctas[i] - 1) / ctas[i]);
  }
  const Cuts c{before.data(), front.data(), ctas.data(), n_tiles, h_kv, equal_costs(total, n_tiles * h_kv, n_ctas),
               own_pieces(front[n_tiles], n_ctas, longest, equal_blocks(total, n_ctas))};
  for (unsigned b = 0; b <= n_ctas; ++b) cuts[b] = c.cut(b, units[b]);
  for (unsigned u = 0; u < n_tiles * h_kv; ++u) c.ctas_of(u, by[2 * u], by[2 * u + 1]);
  return c.own;
}
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    where = tmp_path_factory.mktemp("cuts")
    (where / "cuts.cpp").write_text(SOURCE)
    subprocess.run(["g++", "-O2", "-shared", "-fPIC", "-std=c++17", "-I", os.path.join(PKG_DIR, "csrc"), "-o", str(where / "cuts.so"),
                    str(where / "cuts.cpp")], check=True, timeout=120)
    lib = ctypes.CDLL(str(where / "cuts.so"))

    def run(lens, h_kv, n_ctas):
        U = ctypes.c_uint32
        cuts, units = (U * (n_ctas + 1))(), (U * (n_ctas + 1))()
        by = (ctypes.c_int * (2 * len(lens) * h_kv))()
        own = lib.plan((U * len(lens))(*lens), len(lens), h_kv, n_ctas, cuts, units, by)
        return list(cuts), list(units), [(by[2 * u], by[2 * u + 1]) for u in range(len(lens) * h_kv)], bool(own)

    return run


def _check(plan, lens, h_kv, n_ctas):
    cuts, units, by, own = plan(lens, h_kv, n_ctas)
    what = (lens, h_kv, n_ctas, own)
    starts = [0]
    for n in lens:
        starts += [starts[-1] + n * (i + 1) for i in range(h_kv)]
    total = starts[-1]
    assert cuts[0] == 0 and cuts[n_ctas] == total and all(a <= b for a, b in zip(cuts, cuts[1:])), what
    owners, begun = [[] for _ in by], [0] * n_ctas
    for b in range(n_ctas):
        # as a CTA walks: from the unit that its cut names on, up to the next cut
        u, a, e = units[b], cuts[b], cuts[b + 1]
        assert a == e or starts[u] <= a < starts[u + 1], what
        while u < len(by) and starts[u] < e:
            assert min(e, starts[u + 1]) > max(a, starts[u]), what
            begun[b] += starts[u] >= a
            owners[u].append(b)
            u += 1
    for u, (first, last) in enumerate(by):
        assert owners[u] == list(range(first, last + 1)) and last < n_ctas, (what, u, first, last, owners[u])
    # no CTA gets many units of its own while others have one: a unit costs it four blocks and more
    cost = [4 * n + e - a for n, a, e in zip(begun, cuts, cuts[1:])]
    assert own or max(cost) <= max(6, -(-(total + 4 * len(by)) // n_ctas)) + 4, (what, max(cost))
    return own


@pytest.mark.parametrize("lens", [[128, 2, 2], [2, 2, 128], [128, 4, 4, 4, 4], [256, 8, 8, 8], [8, 8, 8, 256], [128, 1, 1], [1, 1, 128],
                                  [64, 2, 2], [128, 1], [1], [2], [1, 1], [1, 1, 1], [3], [1000] + [1] * 30, [128, 2, 2, 2, 2, 2, 2, 2]], ids=str)
@pytest.mark.parametrize("h_kv", [1, 2, 8])
@pytest.mark.parametrize("n_ctas", [148, 152, 160])
def test_every_block_has_one_cta(plan, lens, h_kv, n_ctas):
    _check(plan, lens, h_kv, n_ctas)


def test_ragged_lengths(plan):
    rng = random.Random(1)
    kinds = [0, 0]
    for _ in range(4000):
        h_kv, n = rng.choice([1, 2, 3, 4, 8]), rng.randint(1, 40)
        most = 2 ** rng.uniform(0, 11)
        lens = [max(1, int(most ** rng.random())) for _ in range(n)]
        rng.shuffle(lens)
        kinds[_check(plan, lens, h_kv, rng.choice([148, 152]))] += 1
    assert min(kinds) > 200, kinds


def test_the_largest_lengths(plan):
    # 2^24 blocks of a tile, and 2^30 of all, is what the plan's 32 bits are for
    for lens, h_kv in (([1 << 24], 1), ([1 << 24, 1], 8), ([1, 1 << 24, 77], 16), ([(1 << 24) - 1] * 7, 8)):
        _check(plan, lens, h_kv, 152)
