"""Raw tail rows of the packed cache that are not finite: a value reaches its channel, as in decode attention,
and a key every row."""
import pytest
import torch

from cache_util import Cache
from test_gpu_tree import Drafts, _call

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("q_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,batch", [(1, 3), (4, 3), (10, 3), (10, 60), (10, 150), (30, 150)])
@pytest.mark.parametrize("bits,B", [(2, 32), (4, 64)])
def test_tail_rows_that_are_not_finite(kvlib, bits, B, T, batch, q_dtype):
    kv = kvlib
    lens = [3 * B + B - 1, 21, 2 * B] + [B + 5] * (batch - 3)
    c = Cache(kv, 95, lens, 8, 2, B, bits)
    d = Drafts(c, T, q_dtype=q_dtype)
    want = _call(c, d)
    c.staging[0, 1, 1, 17, 5] = float("inf")
    c.staging[1, 0, 1, 20, 77] = float("nan")
    out = _call(c, d)
    hit = torch.zeros(batch, T, 8, 128, dtype=torch.bool, device="cuda")
    hit[0, :, 4:, 5] = True                     # kv head 1: query heads 4 .. 7
    hit[1, :, :4, 77] = True
    assert torch.equal(~torch.isfinite(out), hit)
    assert torch.equal(out[~hit], want[~hit])
    # decode attention over the same cache: the same channels
    one, ws = torch.zeros(batch, 8, 128, device="cuda"), kv.alloc_workspace(c.cfg, batch, c.table.shape[1])
    kv.decode_attn(c.cfg, d.q[:, 0].contiguous(), c.pool, c.staging, c.table, c.seq_lens, one, ws)
    assert torch.equal(~torch.isfinite(one), hit[:, 0])
    c.staging[0, 1, 0, 3, 9] = float("nan")     # a key
    out = _call(c, d)
    hit[0, :, 4:] = True
    assert torch.equal(~torch.isfinite(out), hit)
    assert torch.equal(out[~hit], want[~hit])
