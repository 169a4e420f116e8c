"""The insert into the paged 8-bit cache where values are not finite.  Cache and its helpers are those of
test_kv8_insert_gpu: codes and scales agree with the oracle bit for bit."""

import numpy as np
import pytest
import torch

from test_kv8_insert_gpu import Cache, _slots, _values

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from top_sparse_mla_gb300 import native
    from top_sparse_mla_gb300.build import build
    build()
    native.library()


@pytest.mark.parametrize("what", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_one_value_leaves_its_page_and_scale_as_they_are(what, dtype):
    page, h, d = 16, 2, 64
    one, other = Cache(20, 4, h, page, d), Cache(20, 4, h, page, d)
    k = _values(21, 3, h, d, dtype, spread=0.0)
    bad = k.clone()
    bad[1, 1, 7] = what
    slots = np.array([37, 38, 39])   # page 2, behind five older rows
    for c, x in ((one, k), (other, bad)):
        c.insert(x, x, slots)
    for a, b in zip(one.dev, other.dev):
        diff = (a != b).nonzero()
        assert len(diff) <= 1 and (len(diff) == 0 or diff[0].tolist() == [2, 1, 6, 7])
    assert other.dev[0][2, 1, 6, 7].item() == {float("inf"): 0x7E, float("-inf"): 0xFE}.get(what, 0x7F)


@pytest.mark.parametrize("d,page", [(64, 16), (128, 32), (64, 128), (128, 64)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_values_that_are_not_finite_in_ragged_requests(d, page, dtype):
    """Infinities and NaNs of both signs among the values, some tokens of nothing else, and runs of nothing but infinities."""
    h = 3
    lens = [(0, 1), (page - 1, 1), (5, 2 * page + 3), (page, 1), (page // 2, page // 2), (3, 70), (0, 191), (7, 1)]
    n = sum(b for _, b in lens)
    cache = Cache(page + d + 1, 60, h, page, d)
    slots = _slots(page, lens, page, 60, pad=3)
    rng = np.random.default_rng(d)

    def values(seed):
        x = _values(seed, n + 3, h, d, dtype)
        for what, share in ((float("inf"), 0.002), (float("-inf"), 0.002), (float("nan"), 0.002)):
            x[torch.from_numpy(rng.random(tuple(x.shape)) < share).cuda()] = what
        x[4], x[-9:-6], x[0, 1] = float("nan"), float("inf"), float("-inf")
        return x

    cache.insert(values(22), values(23), slots)
    cache.insert(values(24), values(25), slots)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_maxima_at_every_exponent_of_the_type(dtype):
    """Runs whose largest magnitude is 2^e, 1.75 * 2^e or just above, down to the type's subnormals."""
    page, h, d = 16, 1, 64
    low, high = (-133, 127) if dtype == "bf16" else (-24, 15)
    values = [m * 2.0 ** e for e in range(low, high + 1) for m in (1.0, 1.75, 1.7578125) if m * 2.0 ** e < 2.0 ** (high + 1)]
    n = len(values)
    cache = Cache(26, n, h, page, d)
    k = torch.zeros((n, h, d), dtype=torch.float64)
    k[:, 0, 0], k[:, 0, 1] = torch.tensor(values, dtype=torch.float64), -torch.tensor(values, dtype=torch.float64) / 3
    k = k.to(torch.bfloat16 if dtype == "bf16" else torch.float16).cuda()
    assert not k.isinf().any()
    cache.insert(k, -k, np.arange(n) * page)
