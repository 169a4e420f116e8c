"""The insert into the paged 8-bit cache (include/dsa_kv8.h) against the oracle
(oracle/paged.py).  Scales are powers of two, so every product is exact on both sides and
codes and scales agree bit for bit; every other byte of the pools stays as it was."""

import numpy as np
import pytest
import torch

from oracle import paged
from top_sparse_mla_gb300 import native

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from top_sparse_mla_gb300.build import build
    build()
    native.library()


class Cache:
    """Pools of random bytes (finite codes) with power-of-two scales, and the oracle's copy."""

    def __init__(self, seed, n_pages, h, page, d):
        rng = np.random.default_rng(seed)
        self.page = page
        self.ref = []
        for _ in range(2):
            pool = rng.integers(0, 256, (n_pages, h, page, d)).astype(np.uint8)
            pool[(pool & 0x7F) == 0x7F] = 0x11
            scale = np.exp2(rng.integers(-12, 2, (n_pages, h))).astype(np.float32)
            self.ref += [pool, scale]
        self.dev = [torch.from_numpy(x.copy()).cuda() for x in self.ref]

    def insert(self, k, v, slots, status=None, reference=True):
        """k, v: device tensors; both sides, then compared."""
        kp, ks, vp, vs = self.dev
        native.dsa_kv8_insert(k, v, torch.from_numpy(np.asarray(slots, np.int64)).cuda(), kp, vp, ks, vs, status=status)
        torch.cuda.synchronize()
        if reference:
            for i, x in ((0, k), (2, v)):
                self.ref[i], self.ref[i + 1] = paged.kv8_insert(self.ref[i], self.ref[i + 1], x.double().cpu().numpy(), slots)
        self.compare()

    def compare(self):
        for name, got, want in zip(("k codes", "k scales", "v codes", "v scales"), self.dev, self.ref):
            g = got.cpu().numpy()
            assert np.array_equal(g, want), f"{name}: {int((g != want).sum())} of {g.size} differ"


def _values(seed, n, h, d, dtype, spread=3.0):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn((n, h, d), generator=gen) * torch.exp2(torch.randn((n, h, 1), generator=gen) * spread)
    return x.to(TYPES[dtype]).cuda()


def _slots(seed, lens, page, n_pages, pad=0):
    """Slots of requests (before, new) on pages of a random order, and `pad` skipped rows behind them."""
    ids = np.random.default_rng(seed).permutation(n_pages)
    out, at = [], 0
    for before, new in lens:
        p = np.arange(before, before + new)
        out.append(ids[at + p // page] * page + p % page)
        at += -(-(before + new) // page)
    assert at <= n_pages
    return np.concatenate(out + [np.full(pad, -1)]).astype(np.int64)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_ragged_requests(d, page, dtype):
    h = 3
    lens = [(0, 1), (page - 1, 1), (5, 2 * page + 3), (0, 0), (page, 1), (page // 2, page // 2), (3, 70), (0, 191), (7, 1)]
    n = sum(b for _, b in lens)
    cache = Cache(page + d, 60, h, page, d)
    slots = _slots(page, lens, page, 60, pad=3)
    cache.insert(_values(1, n + 3, h, d, dtype), _values(2, n + 3, h, d, dtype), slots)


@pytest.mark.parametrize("n", [1, 63, 64, 65, 300])
def test_one_token_per_request(n):
    page, h, d = 64, 2, 128
    rng = np.random.default_rng(n)
    cache = Cache(n, n, h, page, d)
    for step in range(2):
        slots = rng.permutation(n) * page + rng.integers(0, page - 2, n) + step
        if step == 0:
            slots[::7] = -1
        cache.insert(_values(10 * n + step, n, h, d, "bf16"), _values(10 * n + 5 + step, n, h, d, "bf16"), slots)


def test_pages_filled_in_pieces_match_pages_filled_at_once():
    page, h, d = 64, 2, 128
    gen = torch.Generator().manual_seed(3)
    # values of at least 2^-6 of any scale of the page: no piece rounds below the normal range
    k = ((torch.rand((2 * page, h, d), generator=gen) + 0.02) * 64).to(torch.bfloat16).cuda()
    one, many = Cache(4, 4, h, page, d), Cache(4, 4, h, page, d)
    slots = np.concatenate([page + np.arange(page), 3 * page + np.arange(page)])
    one.insert(k, -k, slots)
    for a, b in ((0, 1), (1, 2), (2, 40), (40, 100), (100, 128)):
        many.insert(k[a:b], -k[a:b], slots[a:b])
    for x, y in zip(one.dev, many.dev):
        assert torch.equal(x, y)


def test_growing_scales_rescale_the_older_rows():
    page, h, d = 32, 2, 64
    cache = Cache(6, 8, h, page, d)
    for step in range(page):   # every token doubles the magnitude
        k = _values(step, 8, h, d, "bf16", spread=0.0) * 2.0 ** (step - 20)
        cache.insert(k, k * 0.5, np.arange(8) * page + step)


def test_extreme_magnitudes():
    page, h, d = 16, 2, 64
    cache = Cache(7, 6, h, page, d)
    k = _values(8, 12, h, d, "bf16", spread=0.0)
    k[0] = 0.0                      # an all-zero run
    k[1] *= 2.0 ** -100             # below the least scale: zeros
    k[2] = 448.0                    # exactly at a scale's end, and just past it
    k[3] = 450.0
    k[4] = 3.0e38                   # past the largest scale: saturates
    k[5] *= 2.0 ** 60
    k[6] = -448.0 * 2.0 ** 64
    slots = np.array([0, 16, 32, 48, 64, 80 + 3, 80 + 4, 80 + 5, 1, 17, 33, 49])
    for a, b in ((0, 8), (8, 12)):   # the second call continues pages of the first
        cache.insert(k[a:b], k.flip(0)[a:b], slots[a:b])


def test_non_finite_values_stay_in_their_page():
    page, h, d = 16, 1, 64
    cache = Cache(9, 4, h, page, d)
    before = [x.cpu().numpy().copy() for x in cache.dev]
    k = torch.ones((3, h, d), dtype=torch.float16, device="cuda")
    k[0, 0, 5] = float("inf")
    k[1, 0, 7] = float("nan")
    kp, ks, vp, vs = cache.dev
    native.dsa_kv8_insert(k, k, torch.tensor([3, 32, 33], device="cuda"), kp, vp, ks, vs)
    assert kp[0, 0, 3, 5].item() == 0x7E            # an infinity saturates
    assert (kp[2, 0, 0, 7].item() & 0x7F) == 0x7F   # the NaN code
    assert ks[2, 0].item() == 2.0 ** -8             # the NaN does not change the scale of 1.0s
    for i in (0, 2):
        assert np.array_equal(cache.dev[i][1].cpu().numpy(), before[i][1])
        assert np.array_equal(cache.dev[i][3].cpu().numpy(), before[i][3])


def test_strided_keys_and_values():
    page, h, d, n = 16, 3, 64, 40
    gen = torch.Generator().manual_seed(4)
    packed = torch.randn((n, 2 * h + 2, d), generator=gen).to(torch.bfloat16).cuda()     # one projection's output
    slots = _slots(5, [(3, 40)], page, 9)
    Cache(10, 9, h, page, d).insert(packed[:, 1:1 + h], packed[:, 1 + h:1 + 2 * h], slots)
    heads_first = torch.randn((h, n, d), generator=gen).to(torch.float16).cuda()
    Cache(11, 9, h, page, d).insert(heads_first.transpose(0, 1), heads_first.flip(0).transpose(0, 1), slots)
    one = torch.randn((n, 2, d), generator=gen).to(torch.float16).cuda()                  # one head of two
    Cache(12, 9, 1, page, d).insert(one[:, 1:], one[:, :1], slots)


def test_slots_out_of_range_are_skipped_and_reported():
    page, h, d = 16, 2, 64
    cache = Cache(13, 4, h, page, d)
    k = _values(14, 6, h, d, "fp16")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    slots = np.array([5, 64, 2 ** 40, 17, 18, -2 ** 40])
    cache.insert(k, k, slots, status=status)
    assert status.item() == native.DSA_STATUS_SLOT_OUT_OF_RANGE
    status.zero_()
    cache.insert(k[:1], k[:1], np.array([63]), status=status)
    assert status.item() == 0


def test_pools_past_32_bits_and_many_heads():
    # a pool of 2.2 GB: the last pages lie past 2^31 bytes
    page, h, d, n_pages = 128, 16, 128, 8448
    pools = [torch.zeros((n_pages, h, page, d), dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.ones((n_pages, h), device="cuda") for _ in range(2)]
    k = _values(15, 130, h, d, "bf16")
    slots = np.arange((n_pages - 2) * page + 5, (n_pages - 2) * page + 135)
    native.dsa_kv8_insert(k, -k, torch.from_numpy(slots).cuda(), pools[0], pools[1], scales[0], scales[1])
    torch.cuda.synchronize()
    for pool, scale, x in ((pools[0], scales[0], k), (pools[1], scales[1], -k)):
        want, ws = paged.kv8_insert(np.zeros((2, h, page, d), np.uint8), np.ones((2, h), np.float32), x.double().cpu().numpy(),
                                    slots - (n_pages - 2) * page)
        assert np.array_equal(pool[-2:].cpu().numpy(), want) and np.array_equal(scale[-2:].cpu().numpy(), ws)
        assert int(pool[:-2].max()) == 0 and (scale[:-2] == 1).all()


def test_repeated_and_replayed_calls_change_nothing():
    page, h, d = 64, 2, 128
    lens = [(10, 30), (63, 2), (0, 129)]
    cache = Cache(16, 12, h, page, d)
    n = sum(b for _, b in lens)
    k, v, slots = _values(17, n, h, d, "bf16"), _values(18, n, h, d, "bf16"), _slots(19, lens, page, 12)
    cache.insert(k, v, slots)
    cache.insert(k, v, slots, reference=False)   # the same tokens again: the same pages
    kp, ks, vp, vs = cache.dev
    sl = torch.from_numpy(slots).cuda()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        native.dsa_kv8_insert(k, v, sl, kp, vp, ks, vs)
    graph.replay()
    torch.cuda.synchronize()
    cache.compare()
