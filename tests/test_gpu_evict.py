"""Eviction by accumulated weights against a selection by sorting: what is kept is
moved as it is, so that everything has to be equal."""
import numpy as np
import pytest
import torch

from cache_util import Cache, i32

pytestmark = pytest.mark.gpu


def _want(c, weights, budget, recent, new_blocks, lens=None):
    """(new_lens, kept, new_weights) by the definition."""
    w = weights.cpu().numpy()
    batch, n_kv, B = len(c.lens), c.n_kv, c.B
    unit = B if c.bits else 1
    places, last = budget // unit, recent // unit
    kept = np.full((batch, n_kv, places), -1, np.int32)
    new_w = np.zeros((batch, n_kv, new_blocks * B), np.float32)
    new_lens = np.zeros(batch, np.int32)
    for b, L in enumerate(c.lens if lens is None else lens):
        have = L // unit
        size = min(have, places)
        new_lens[b] = size * unit + L % unit
        for h in range(n_kv):
            x = w[b, h, :have * unit].reshape(have, unit).astype(np.float64)
            x = np.where(x > 0, x, 0.0).sum(1).astype(np.float32)
            pick = np.arange(have)
            if have > places:
                old = have - last
                best = np.lexsort((np.arange(old), -x[:old].astype(np.float64)))[:places - last]
                pick = np.concatenate([np.sort(best), np.arange(old, have)]).astype(int)
            kept[b, h, :size] = pick
            t = np.concatenate([(pick[:, None] * unit + np.arange(unit)).ravel(), np.arange(have * unit, L)]).astype(int)
            new_w[b, h, :len(t)] = w[b, h, t]
    return new_lens, kept, new_w


def _run(c, weights, budget, recent, new_blocks=None, new_table=None, lens=None, ws=None, check=True):
    kv = c.kv
    batch, n_kv, B = len(c.lens), c.n_kv, c.B
    new_blocks = budget // B + 1 if new_blocks is None else new_blocks
    new_table = torch.from_numpy(c.spare_np[:batch * new_blocks].reshape(batch, new_blocks)).cuda() if new_table is None else new_table
    places = budget // B if c.bits else budget
    new_lens = torch.full((batch,), 99, dtype=torch.int32, device="cuda")
    new_w = torch.full((batch, n_kv, new_blocks * B), 5.0, device="cuda")
    kept = torch.full((batch, n_kv, places), 77, dtype=torch.int32, device="cuda")
    ws = kv.alloc_workspace(c.cfg, 0, 0) if ws is None else ws
    call = kv.evict if c.bits else kv.evict_bf16
    call(c.cfg, c.pool, c.table, c.seq_lens if lens is None else lens, weights, new_table, new_lens, new_w, kept, ws,
         budget=budget, recent=recent)
    if check:
        assert kv.read_error(ws) == 0
    return new_lens, kept, new_w, new_table


def _rows(c, pool, table, h, n):
    """What the first n places of each sequence of a table hold, kv head h: raw bytes [batch][n][...]."""
    t = table.long()
    if c.bits:
        return pool.view(c.n_pool, c.n_kv, -1)[t[:, :n], h]
    x = pool[t, h].view(torch.int16).transpose(1, 2).flatten(2, 3)      # [batch][2][tokens][128]
    return x[:, :, :n].transpose(1, 2)


def _check(c, weights, budget, recent, new_blocks=None):
    new_blocks = budget // c.B + 1 if new_blocks is None else new_blocks
    before = c.pool.clone()
    new_lens, kept, new_w, new_table = _run(c, weights, budget, recent, new_blocks)
    lens_want, kept_want, w_want = _want(c, weights, budget, recent, new_blocks)
    assert (new_lens.cpu().numpy() == lens_want).all()
    assert (kept.cpu().numpy() == kept_want).all()
    assert (new_w.cpu().numpy().view(np.int32) == w_want.view(np.int32)).all()
    places = kept.shape[2]
    n_old = max(1, c.table.shape[1] * (1 if c.bits else c.B))
    for h in range(c.n_kv):
        got = _rows(c, c.pool, new_table, h, places)
        if c.table.shape[1] == 0:
            continue
        src = _rows(c, before, c.table, h, n_old)
        for b in range(len(c.lens)):
            at = kept[b, h][kept[b, h] >= 0].long()
            assert torch.equal(got[b, :len(at)], src[b, at]), (b, h)
            # behind the new length: as it was
            was = _rows(c, before, new_table[b:b + 1], h, places)[0]
            assert torch.equal(got[b, len(at):], was[len(at):])
    # the old pages are only read
    rest = torch.ones(c.n_pool, dtype=torch.bool, device="cuda")
    rest[new_table.long().flatten()] = False
    as_bytes = lambda p: p.view(torch.uint8) if c.bits else p.view(torch.int16)  # noqa: E731
    assert torch.equal(as_bytes(c.pool)[rest], as_bytes(before)[rest])


def _weights(c, seed, kind):
    g = torch.Generator(device="cuda").manual_seed(seed)
    shape = (len(c.lens), c.n_kv, max(1, c.table.shape[1]) * c.B)
    x = torch.rand(*shape, generator=g, device="cuda")
    if kind == "spread":
        return torch.exp(8 * x - 4) * (x > 0.1)
    if kind == "ties":       # a handful of values, most of them shared
        return torch.floor(4 * x) / 4
    if kind == "equal":
        return torch.full(shape, 0.3, device="cuda")
    if kind == "zero":
        return torch.zeros(shape, device="cuda")
    if kind == "close":      # values that differ in their last bits alone
        return (1 + torch.floor(16 * x) * 2.0 ** -23).contiguous()
    return torch.where(x < 0.2, float("inf"), torch.where(x < 0.4, 3e38, torch.where(x < 0.6, 1e-40, x)))   # extremes


@pytest.mark.parametrize("kind", ["spread", "ties", "equal", "zero", "close", "extremes"])
@pytest.mark.parametrize("bits,B,n_kv", [(0, 32, 3), (0, 64, 1), (2, 32, 2), (2, 64, 3), (3, 32, 1), (4, 64, 2)])
def test_against_a_sort(kvlib, kind, bits, B, n_kv):
    lens = [0, 1, B - 1, B, 3 * B, 3 * B + 1, 7 * B + 5, 300, 16 * B]
    budget, recent = (4 * B, 2 * B) if bits else (3 * B + 7, 19)
    blocks = budget // B + 2
    c = Cache(kvlib, 2, lens, n_kv, n_kv, B, bits, spare=len(lens) * blocks)
    _check(c, _weights(c, 1, kind), budget, recent, blocks)


@pytest.mark.parametrize("bits,budget,recent", [(0, 1, 0), (0, 1, 1), (0, 31, 31), (0, 500, 0), (0, 5000, 7), (2, 32, 0),
                                                (2, 32, 32), (2, 2048, 64), (2, 320, 288)])
def test_budgets(kvlib, bits, budget, recent):
    lens = [1500, 2, 33, 320, 321, 640]
    c = Cache(kvlib, 5, lens, 2, 2, 32, bits, spare=len(lens) * (budget // 32 + 1))
    _check(c, _weights(c, 3, "spread"), budget, recent)


@pytest.mark.parametrize("bits", [0, 2])
@pytest.mark.parametrize("L,budget", [(70000, 4096), (40007, 20032)])
def test_long_sequences(kvlib, bits, L, budget):
    c = Cache(kvlib, 7, [L, 1000], 1, 1, 64, bits, spare=2 * (budget // 64 + 1))
    _check(c, _weights(c, 9, "spread"), budget, 128)
    _check(c, _weights(c, 9, "ties"), budget, 0)


def test_places_beyond_four_gigabytes(kvlib):
    c = Cache(kvlib, 9, [300, 77], 2, 2, 64, 0, extra=70000, spare=8)
    assert int(c.table.min()) * 2 * 2 * 64 * 128 * 2 > 1 << 32
    w = _weights(c, 2, "spread")
    new_lens, kept, new_w, new_table = _run(c, w, 128, 16)
    want = _want(c, w, 128, 16, 3)
    assert (kept.cpu().numpy() == want[1]).all() and (new_lens.cpu().numpy() == want[0]).all()
    for h in range(2):
        got, src = _rows(c, c.pool, new_table, h, 128), _rows(c, c.pool, c.table, h, 320)
        assert torch.equal(got[0], src[0, kept[0, h].long()])


def test_pages_shared_by_sequences_are_only_read(kvlib):
    """Two sequences that begin with the same pages, as behind one prompt."""
    c = Cache(kvlib, 12, [256, 256], 2, 2, 32, 0, spare=10)
    c.table[1, :4] = c.table[0, :4]
    _check(c, _weights(c, 4, "spread"), 100, 10)


@pytest.mark.parametrize("bits", [0, 3])
def test_negative_and_missing_weights_count_as_zero(kvlib, bits):
    c = Cache(kvlib, 13, [400, 256], 2, 2, 32, bits, spare=12)
    w = _weights(c, 6, "spread")
    w[:, :, ::3] = -w[:, :, ::3]
    w[:, :, ::7] = float("nan")
    w[:, :, 5::50] = -0.0
    new_lens, kept, _, _ = _run(c, w, 160, 32)
    assert (kept.cpu().numpy() == _want(c, w, 160, 32, 6)[1]).all()


@pytest.mark.parametrize("bits", [0, 2])
def test_graph_replay(kvlib, bits):
    c = Cache(kvlib, 14, [500, 90], 2, 2, 32, bits, spare=12)
    w = _weights(c, 8, "spread")
    want = _run(c, w, 160, 32)
    new_lens, kept, new_w = (torch.zeros_like(x) for x in want[:3])
    ws = c.kv.alloc_workspace(c.cfg, 0, 0)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            (c.kv.evict if bits else c.kv.evict_bf16)(c.cfg, c.pool, c.table, c.seq_lens, w, want[3], new_lens, new_w, kept,
                                                      ws, budget=160, recent=32)
        graph.replay()
        graph.replay()
    side.synchronize()
    for a, b in zip((new_lens, kept, new_w), want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("bits", [0, 2])
def test_faults_are_flagged(kvlib, bits):
    kv = kvlib
    c = Cache(kv, 15, [300, 200, 64], 2, 2, 32, bits, spare=18)
    w = _weights(c, 8, "spread")
    ws = kv.alloc_workspace(c.cfg, 0, 0)
    good = _run(c, w, 160, 32)
    got = _run(c, w, 160, 32, ws=ws, lens=i32([300, -3, 64]), check=False)
    assert kv.read_error(ws) == kv.DEVERR_POSITION
    assert got[0].tolist() == [good[0][0].item(), 0, good[0][2].item()]
    assert (got[1][1] == -1).all() and torch.equal(got[1][0], good[1][0]) and torch.equal(got[2][2], good[2][2])
    kv.clear_error(ws)
    got = _run(c, w, 160, 32, ws=ws, lens=i32([300, c.table.shape[1] * 32 + 1, 64]), check=False)
    assert kv.read_error(ws) == kv.DEVERR_POSITION and got[0][1] == 0
    kv.clear_error(ws)
    bad = good[3].clone()
    bad[1, 0] = -1
    before = c.pool.clone()
    _run(c, w, 160, 32, ws=ws, new_table=bad, check=False)
    assert kv.read_error(ws) == kv.DEVERR_BLOCK_ID
    assert torch.equal(c.pool.view(torch.uint8), before.view(torch.uint8))
    kv.clear_error(ws)
    c.table[0] = c.n_pool
    _run(c, w, 160, 32, ws=ws, check=False)
    assert kv.read_error(ws) == kv.DEVERR_BLOCK_ID


def test_more_blocks_than_shared_memory_holds(kvlib):
    c = Cache(kvlib, 16, [330016, 64], 1, 1, 32, 2, spare=2 * 5001)
    _check(c, _weights(c, 10, "ties"), 5000 * 32, 320)
