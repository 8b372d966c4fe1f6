"""A packed block's weight is the sum of its tokens', rounded to 32 bits as a sum in 64 bits would be: blocks whose
order the last bits of that sum decide."""
import numpy as np
import pytest
import torch

from cache_util import Cache
from test_gpu_evict import _check, _want

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("held", [True, False])
@pytest.mark.parametrize("B", [32, 64])
def test_terms_that_decide_the_rounding(kvlib, B, held):
    """1 + 2^-24 + 2^-50 rounds to 1 + 2^-23 and ties with it; without its last term it rounds to 1. Three budgets: the
    tied blocks that come first are kept. `held`: the keys fit shared memory."""
    blocks = 12 if held else 10240
    c = Cache(kvlib, 80, [blocks * B + 3], 1, 1, B, 2, spare=3 * 9)
    w = np.zeros((1, 1, (blocks + 1) * B), np.float32)
    x = w[0, 0, :blocks * B].reshape(blocks, B)
    r = np.random.default_rng(1)
    for i in range(12):
        terms = ([1.0, 2.0 ** -24, 2.0 ** -50], [1 + 2.0 ** -23], [1.0, 2.0 ** -24])[i % 3]
        x[i, r.permutation(B)[:len(terms)]] = terms
    weights = torch.from_numpy(w).cuda()
    for n, last in ((3, 0), (6, 1), (8, 0)):
        want = _want(c, weights, n * B, last * B, n + 1)[1][0, 0]
        # (of the four with each: 0, 1, 3, 4, 6, 7, 9 and 10 tie above 2, 5, 8 and 11)
        assert list(want[:n - last]) == [0, 1, 3, 4, 6, 7, 9, 10][:n - last]
        _check(c, weights, n * B, last * B)


@pytest.mark.parametrize("kind", ["powers", "wide", "narrow"])
@pytest.mark.parametrize("B", [32, 64])
def test_sums_of_many_sizes(kvlib, B, kind):
    """Blocks that hold the same terms in another order, or all but one of the smallest: their sums tie or are next to one another."""
    blocks, n = 4096, 2000
    c = Cache(kvlib, 81, [blocks * B], 1, 1, B, 3, spare=n + 1)
    r = np.random.default_rng(B)
    if kind == "powers":
        base = 2.0 ** r.integers(-45, 1, (blocks // 8, 1, B))
    elif kind == "wide":
        base = np.exp(r.normal(0, 3, (blocks // 8, 1, B)))
    else:
        base = 1 + r.integers(0, 16, (blocks // 8, 1, B)) * 2.0 ** -23
    x = np.repeat(base, 8, 1).astype(np.float32)
    x[:, 4:, B - 1] = 0
    x = r.permuted(x, axis=2).reshape(blocks, B)
    weights = torch.from_numpy(np.ascontiguousarray(r.permutation(x).reshape(1, 1, -1))).cuda()
    _check(c, weights, n * B, 0)


@pytest.mark.parametrize("B", [32, 64])
def test_infinite_sums(kvlib, B):
    """Weights that are infinite, or whose sum is, beside ones that are not."""
    c = Cache(kvlib, 82, [40 * B], 1, 1, B, 2, spare=21)
    r = np.random.default_rng(2)
    x = r.random((40, B)).astype(np.float32)
    x[3, 5], x[11, :2], x[17], x[30, B - 1] = np.inf, 3e38, 2e38, 3e38
    x[11, 7] = np.nan
    x[20] = -x[20]
    with np.errstate(over="ignore"):
        _check(c, torch.from_numpy(x.reshape(1, 1, -1)).cuda(), 20 * B, 2 * B)
