"""Decode attention with weights beside plain decode attention: the split kernel that leaves its scores fills the GPU
as the plain one does. Its partition is the plain one's, so that a kernel which held fewer CTAs an SM
would run a second wave of part of its warps."""
import pytest
import torch

import synth

pytestmark = pytest.mark.gpu
D = 128


def _times(calls, rounds=12):
    """Least microseconds of each call, taken in turn."""
    best = [float("inf")] * len(calls)
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    for f in calls:
        f()
    for _ in range(rounds):
        for i, f in enumerate(calls):
            start.record()
            for _ in range(4):
                f()
            end.record()
            end.synchronize()
            best[i] = min(best[i], start.elapsed_time(end) * 250)
    return best


@pytest.mark.parametrize("bits,B", [(2, 32), (2, 64), (3, 32), (3, 64), (4, 32), (4, 64)])
def test_a_large_batch(kvlib, bits, B):
    """64 x 8192 tokens. The weights cost 40 bytes a (token, kv head) of 4 query heads: scores written and read, weights read
    and written, 168 MB or 25 us at a copy's 6.78 TB/s, a fifth of the 127 or more that plain decode attention
    takes. A quarter of the warps in a second wave takes a third or more. The bound lies between."""
    kv = kvlib
    batch, L, n_q, n_kv = 64, 8192, 32, 8
    cfg = kv.make_config(n_q, n_kv, B, 2, synth.sign_bits(1), bits=bits)
    nb = L // B
    pool, staging = kv.alloc_pool(cfg, batch * nb), kv.alloc_staging(cfg, batch)
    table = torch.randperm(batch * nb, device="cuda").to(torch.int32).view(batch, nb)
    lens = torch.full((batch,), L, dtype=torch.int32, device="cuda")
    q = torch.randn(batch, n_q, D, device="cuda").to(torch.bfloat16)
    out, w = torch.zeros(batch, n_q, D, device="cuda"), torch.zeros(batch, n_kv, L, device="cuda")
    ws, wws = kv.alloc_workspace(cfg, batch, nb), kv.alloc_weights_workspace(cfg, batch, nb)
    plain, kept = _times([lambda: kv.decode_attn(cfg, q, pool, staging, table, lens, out, ws),
                          lambda: kv.decode_attn_weights(cfg, q, pool, staging, table, lens, out, w, wws)])
    assert kv.read_error(ws) == 0 and kv.read_error(wws) == 0
    assert kept <= 1.3 * plain, (plain, kept)
    print(f"\n{bits} bits, blocks of {B}: {plain:.1f} us, with weights {kept:.1f}")
