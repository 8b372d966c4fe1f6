"""The workspace of tree attention made for the largest call serves every smaller one."""
import itertools

import pytest
import torch

from cache_util import Cache
from test_gpu_tree import Drafts, _call

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n_q,n_kv,B,bits", [(32, 8, 64, 2), (40, 10, 32, 2), (24, 8, 64, 4), (8, 4, 32, 3), (4, 4, 64, 2), (4, 1, 32, 2)])
def test_the_size_grows_with_each_argument(kvlib, n_q, n_kv, B, bits):
    kv = kvlib
    cfg = kv.make_config(n_q, n_kv, B, 2, [0] * 4, bits=bits)
    batches = [0, 1, 2, 3, 4, 7, 16, 61, 62, 63, 64, 100, 300, 1000]
    drafts = [*range(1, 50), 64, 65, 68, 69, 96, 127, 128]
    blocks = [0, 1, 2, 3, 4, 16, 32, 63, 64, 65, 200, 4096]
    size = {a: kv.tree_workspace_bytes(cfg, *a) for a in itertools.product(batches, drafts, blocks)}
    for i, axis in enumerate((batches, drafts, blocks)):
        for a, b in zip(axis, axis[1:]):
            for rest in itertools.product(*(x for k, x in enumerate((batches, drafts, blocks)) if k != i)):
                small, large = (rest[:i] + (v,) + rest[i:] for v in (a, b))
                assert 256 <= size[small] <= size[large], (small, large, size[small], size[large])


@pytest.mark.parametrize("bits", [0, 2, 4])
def test_one_workspace_serves_smaller_calls(kvlib, bits):
    kv = kvlib
    big = Cache(kv, 60, [700] * 40, 8, 8, 32, bits)
    ws = kv.alloc_tree_workspace(big.cfg, 40, 40, big.table.shape[1])
    c = Cache(kv, 61, [640, 33, 90], 8, 8, 32, bits)
    for T in (1, 3, 16, 24, 25, 40):
        d = Drafts(c, T, seed=T, q_dtype=torch.float32 if T == 16 else torch.bfloat16)
        assert torch.equal(_call(c, d, ws=ws), _call(c, d))


def test_a_workspace_for_more_drafts(kvlib):
    """6 drafts of a few sequences, which the few-rows kernel splits over many warps, in the space of 8, which it does not take."""
    kv = kvlib
    c = Cache(kv, 62, [2240, 1000, 64], 32, 8, 32, 2, blocks=70)
    ws = kv.alloc_tree_workspace(c.cfg, 3, 8, 70)
    d = Drafts(c, 6)
    assert torch.equal(_call(c, d, ws=ws), _call(c, d))
