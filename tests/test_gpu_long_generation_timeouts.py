"""The wait-timeout path of the kernels that tree attention with few query rows and decode attention
with weights run over the packed cache."""
import pytest
import torch

from cache_util import Cache
from test_gpu_tree import Drafts, _call

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits,B", [(2, 32), (2, 64), (3, 32), (4, 64)])
@pytest.mark.parametrize("T", [1, 4, 6])
def test_tree_attention_with_few_rows(kvlib, bits, B, T):
    kv = kvlib
    c = Cache(kv, 70, [900, 400, 64], 8, 2, B, bits)
    d = Drafts(c, T)
    ws = kv.alloc_tree_workspace(c.cfg, 3, T, c.table.shape[1])
    good = _call(c, d, ws=ws)
    c.cfg.flags |= kv.FLAG_TEST_WAIT_TIMEOUT
    for _ in range(3):
        _call(c, d, ws=ws, check=False)
        assert kv.read_error(ws) == kv.DEVERR_WAIT_TIMEOUT
        kv.clear_error(ws)
    c.cfg.flags &= ~kv.FLAG_TEST_WAIT_TIMEOUT
    assert torch.equal(_call(c, d, ws=ws), good)


@pytest.mark.parametrize("bits,B", [(2, 32), (4, 64)])
def test_decode_attention_with_weights(kvlib, bits, B):
    kv = kvlib
    c = Cache(kv, 71, [900, 400, 64], 8, 2, B, bits)
    q = torch.randn(3, 8, 128, device="cuda").to(torch.bfloat16)
    ws = kv.alloc_weights_workspace(c.cfg, 3, c.table.shape[1])

    def call():
        out, w = torch.zeros(q.shape, device="cuda"), torch.zeros(3, 2, c.table.shape[1] * B, device="cuda")
        kv.decode_attn_weights(c.cfg, q, c.pool, c.staging, c.table, c.seq_lens, out, w, ws, decay=0.0)
        return out, w

    good = call()
    assert kv.read_error(ws) == 0
    c.cfg.flags |= kv.FLAG_TEST_WAIT_TIMEOUT
    for _ in range(3):
        call()
        assert kv.read_error(ws) == kv.DEVERR_WAIT_TIMEOUT
        kv.clear_error(ws)
    c.cfg.flags &= ~kv.FLAG_TEST_WAIT_TIMEOUT
    again = call()
    assert kv.read_error(ws) == 0 and torch.equal(again[0], good[0]) and torch.equal(again[1], good[1])
