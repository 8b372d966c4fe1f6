"""Eviction right behind the kernel that writes its weights, beside whose end it may start."""
import pytest
import torch

from cache_util import Cache

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits,B", [(0, 64), (2, 32), (2, 64)])
def test_weights_written_just_before(kvlib, bits, B):
    """Decode attention with weights and the eviction by them, in turn and as a graph, with another query each time:
    what is kept is what a call gives that waits for everything before it."""
    kv = kvlib
    lens = [3000, 0, 900, 64, 2500, 2999]
    budget, recent = 8 * B, 2 * B
    new_blocks = budget // B + 1
    c = Cache(kv, 97, lens, 8, 2, B, bits, spare=len(lens) * new_blocks)
    batch, blocks = c.table.shape
    ws = kv.alloc_weights_workspace(c.cfg, batch, blocks)
    new_table = torch.from_numpy(c.spare_np.reshape(batch, new_blocks)).cuda()
    w = torch.zeros(batch, 2, blocks * B, device="cuda")
    out = torch.zeros(batch, 8, 128, device="cuda")
    new_lens = torch.zeros(batch, dtype=torch.int32, device="cuda")
    new_w = torch.zeros(batch, 2, new_blocks * B, device="cuda")
    kept = torch.zeros(batch, 2, budget // B if bits else budget, dtype=torch.int32, device="cuda")
    q = torch.zeros(batch, 8, 128, device="cuda")

    def step(wait):
        if bits:
            kv.decode_attn_weights(c.cfg, q, c.pool, c.staging, c.table, c.seq_lens, out, w, ws, decay=0.0)
        else:
            kv.decode_attn_weights_bf16(c.cfg, q, c.pool, c.table, c.seq_lens, out, w, ws, decay=0.0)
        if wait:
            torch.cuda.synchronize()
        (kv.evict if bits else kv.evict_bf16)(c.cfg, c.pool, c.table, c.seq_lens, w, new_table, new_lens, new_w, kept, ws,
                                              budget=budget, recent=recent)

    g = torch.Generator(device="cuda").manual_seed(4)
    queries = [3 * torch.randn(q.shape, generator=g, device="cuda") for _ in range(12)]
    want = []
    for x in queries:
        q.copy_(x)
        step(True)
        want.append((kept.clone(), new_w.clone(), new_lens.clone()))
    assert not torch.equal(want[0][0], want[1][0])
    for x, e in zip(queries, want):
        q.copy_(x)
        step(False)
        assert all(torch.equal(a, b) for a, b in zip((kept, new_w, new_lens), e))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step(False)
        for x, e in zip(queries, want):
            q.copy_(x)
            graph.replay()
            assert all(torch.equal(a, b) for a, b in zip((kept, new_w, new_lens), e))
    side.synchronize()
    assert kv.read_error(ws) == 0
