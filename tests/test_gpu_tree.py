"""Attention for a tree of drafted tokens against softmax in 64 bits over the same
cache bytes (tolerances: cache_util)."""
import numpy as np
import pytest
import torch

import bit_kv_cache_08_gb300 as kv_
from cache_util import Cache, attend, close_rows, i32

pytestmark = pytest.mark.gpu
D = 128


class Drafts:
    """Queries, keys and values of `T` drafts a sequence; k and v columns of one projection's rows."""

    def __init__(self, c, T, seed=0, q_dtype=torch.bfloat16, parents="tree", lens=None, pad=0):
        batch, n_q, n_kv = len(c.lens), c.cfg.n_q_heads, c.n_kv
        g = torch.Generator(device="cuda").manual_seed(seed + 100)
        self.T = T
        self.q = (2 * torch.randn(batch, T, n_q, D, generator=g, device="cuda")).to(q_dtype)
        rows = torch.randn(batch, T, 2 * n_kv * D + pad, generator=g, device="cuda").to(torch.bfloat16)
        self.rows = rows
        self.k = rows[..., :n_kv * D].unflatten(-1, (n_kv, D))
        self.v = rows[..., pad + n_kv * D:].unflatten(-1, (n_kv, D))
        r = np.random.default_rng(seed)
        if parents == "chain":
            self.parents = np.tile(np.arange(-1, T - 1), (batch, 1))
        else:
            self.parents = np.stack([[-1 if i == 0 else int(r.integers(max(-1, i - 9), i)) for i in range(T)] for _ in range(batch)])
        self.mask = kv_.tree_mask(self.parents).cuda()
        self.lens = None if lens is None else i32(lens)

    def shown(self):
        """[batch][T][T] of the mask's bits."""
        w = self.mask.cpu().numpy().view(np.uint32)
        return (w[..., None] >> np.arange(32, dtype=np.uint32) & 1).astype(bool).reshape(*w.shape[:2], -1)[..., :self.T]


def _call(c, d, out_dtype=torch.float32, ws=None, lens=None, out=None, check=True):
    kv = c.kv
    out = torch.full(d.q.shape, 3.0, dtype=out_dtype, device="cuda") if out is None else out
    ws = kv.alloc_tree_workspace(c.cfg, d.q.shape[0], d.T, c.table.shape[1]) if ws is None else ws
    rest = (c.table, c.seq_lens if lens is None else lens, d.k, d.v, d.mask, out, ws)
    if c.bits:
        kv.tree_attn(c.cfg, d.q, c.pool, c.staging, *rest, draft_lens=d.lens)
    else:
        kv.tree_attn_bf16(c.cfg, d.q, c.pool, *rest, draft_lens=d.lens)
    if check:
        assert kv.read_error(ws) == 0
    return out


def _check(c, d, out, seqs=None, rows=None):
    """Sequences (and draft rows) of a call's output; returns the worst error of its bound."""
    n_kv, G, T = c.n_kv, c.cfg.n_q_heads // c.n_kv, d.T
    shown, worst = d.shown(), 0.0
    bf16 = out.dtype is torch.bfloat16
    for b in range(len(c.lens)) if seqs is None else seqs:
        n = T if d.lens is None else int(d.lens[b])
        assert (out[b, n:] == 3.0).all(), "padding rows"
        pick = np.arange(n) if rows is None else np.array([r for r in rows if r < n], int)
        if not len(pick):
            continue
        q, k, v, o = (x[b].double().cpu().numpy() for x in (d.q, d.k, d.v, out))
        for h in range(n_kv):
            (K, V), (ek, ev) = c.tokens(b, h)
            K, V = np.concatenate([K, k[:n, h]]), np.concatenate([V, v[:n, h]])
            ek = np.concatenate([ek, np.linalg.norm(k[:n, h], axis=1)])
            ev = np.concatenate([ev, np.linalg.norm(v[:n, h], axis=1)])
            see = np.concatenate([np.ones((len(pick), c.lens[b]), bool), shown[b][pick][:, :n]], 1).repeat(G, 0)
            want, tol, _, _ = attend(q[pick][:, h * G:(h + 1) * G].reshape(-1, D), K, V, ek, ev, c.scale,
                                     d.q.dtype is torch.float32, see)
            worst = max(worst, close_rows(o[pick][:, h * G:(h + 1) * G].reshape(-1, D), want, tol, bf16))
    return worst


CACHES = [(0, 32, 8, 2), (0, 64, 3, 1), (2, 32, 8, 2), (2, 64, 6, 2), (3, 64, 4, 4), (3, 32, 12, 4), (4, 64, 8, 2), (4, 32, 2, 1)]


@pytest.mark.parametrize("bits,B,n_q,n_kv", CACHES)
@pytest.mark.parametrize("T", [1, 5, 33])
def test_against_64_bits(kvlib, bits, B, n_q, n_kv, T):
    lens = [0, 1, B - 1, B, B + 1, 5 * B + 7, 313, 2]
    c = Cache(kvlib, 11 + bits, lens, n_q, n_kv, B, bits)
    d = Drafts(c, T, seed=T, lens=[T, 0, 1, T, max(1, T - 1), T, T // 2, T], pad=8)
    _check(c, d, _call(c, d))
    _check(c, d, _call(c, d, torch.bfloat16))


@pytest.mark.parametrize("bits,B,n_q,n_kv", CACHES[::2])
@pytest.mark.parametrize("T", [2, 17, 64])
def test_fp32_queries(kvlib, bits, B, n_q, n_kv, T):
    c = Cache(kvlib, 30 + bits, [200, 0, 65], n_q, n_kv, B, bits, sm_scale=0.11)
    d = Drafts(c, T, q_dtype=torch.float32, parents="chain")
    _check(c, d, _call(c, d))


@pytest.mark.parametrize("bits", [0, 2, 4])
@pytest.mark.parametrize("T,n_q", [(31, 4), (32, 4), (33, 4), (64, 4), (65, 2), (96, 3), (128, 4), (128, 1)])
def test_every_number_of_row_tiles(kvlib, bits, T, n_q):
    c = Cache(kvlib, 40, [517, 90], n_q, 1, 64, bits)
    d = Drafts(c, T, seed=2, parents="chain")
    _check(c, d, _call(c, d))


@pytest.mark.parametrize("bits", [0, 2])
@pytest.mark.parametrize("batch,ctx,T", [(1, 20000, 8), (3, 5000, 40), (40, 700, 16), (150, 90, 4)])
def test_few_long_and_many_short_sequences(kvlib, bits, batch, ctx, T):
    lens = np.random.default_rng(batch).integers(ctx // 2, ctx + 1, batch)
    c = Cache(kvlib, 3, lens, 8, 2, 64, bits, wild=batch == 40)
    d = Drafts(c, T, seed=1)
    _check(c, d, _call(c, d), seqs=range(0, batch, 1 + batch // 4), rows=[0, 3, T // 2, T - 1])


@pytest.mark.parametrize("bits", [0, 2])
def test_a_chain_is_decode_attention_over_the_appended_tokens(kvlib, bits):
    """The last row of a chain sees what a decode step sees once its drafts are in the cache."""
    kv = kvlib
    T = 6
    c = Cache(kv, 17, [69, 40, 128], 8, 2, 32, bits, blocks=6)
    d = Drafts(c, T, parents="chain")
    out = _call(c, d)
    ws = kv.alloc_workspace(c.cfg, 3, 6)
    rope = kv.make_rope([])
    k, v = (x.reshape(3 * T, 2, D) for x in (d.k, d.v))
    cu = i32([0, T, 2 * T, 3 * T])
    want = torch.empty(3, 8, D, device="cuda")
    last = d.q[:, -1].contiguous()
    if bits:
        kv.append_rope(c.cfg, rope, c.pool, c.staging, c.table, c.seq_lens, None, k, v, None, ws, cu_tokens=cu)
        kv.decode_attn(c.cfg, last, c.pool, c.staging, c.table, c.seq_lens + T, want, ws)
    else:
        kv.append_rope_bf16(c.cfg, rope, c.pool, c.table, c.seq_lens, None, k, v, None, ws, cu_tokens=cu)
        kv.decode_attn_bf16(c.cfg, last, c.pool, c.table, c.seq_lens + T, want, ws)
    assert kv.read_error(ws) == 0
    # (no sequence completes a block on the way, so that the packed cache holds the drafts unquantised too)
    assert (out[:, -1] - want).norm(dim=-1).max() <= 2.0 ** -13 * want.norm(dim=-1).max()


@pytest.mark.parametrize("bits", [0, 2])
def test_any_mask(kvlib, bits):
    """Rows that see nothing of the tree, all of it, or others' drafts; bits beyond the sequence's drafts are ignored."""
    c = Cache(kvlib, 18, [50, 0, 64, 0], 8, 2, 32, bits)
    d = Drafts(c, 40, lens=[40, 40, 37, 3])
    r = np.random.default_rng(1)
    words = r.integers(0, 2 ** 32, d.mask.shape, dtype=np.uint64).astype(np.uint32)
    words[:, 0] = 0
    words[:, 1] = 0xffffffff
    words[:, 2, 0], words[:, 2, 1] = 0, 1 << 31          # a bit beyond the drafts alone
    d.mask = torch.from_numpy(words.view(np.int32)).cuda()
    out = _call(c, d)
    _check(c, d, out)
    assert (out[1, 0] == 0).all() and (out[1, 2] == 0).all() and (out[3, 0] == 0).all() and (out[3, 2] == 0).all()


@pytest.mark.parametrize("bits", [0, 2])
@pytest.mark.parametrize("T", [7, 48])
def test_values_that_are_not_finite(kvlib, bits, T):
    """A draft that is not finite reaches the rows that see it and no other; padding rows may hold anything."""
    c = Cache(kvlib, 19, [100, 33, 64], 8, 2, 32, bits)
    clean = Drafts(c, T, lens=[T, T, T - 2])
    want = _call(c, clean)
    d = Drafts(c, T, lens=[T, T, T - 2])
    d.rows[2, T - 2:] = float("nan")
    d.q[2, T - 2:] = float("nan")
    d.v[0, 3, 1, 5] = float("inf")
    d.k[0, 5, 0, 9] = float("nan")
    d.q[1, 2, 3, 7] = float("nan")
    out = _call(c, d)
    shown = d.shown()
    hit = torch.zeros(3, T, 8, dtype=torch.bool)
    hit[0, torch.from_numpy(shown[0, :, 3]), 4:] = True       # kv head 1: query heads 4 .. 7
    hit[0, torch.from_numpy(shown[0, :, 5]), :4] = True
    hit[1, 2, 3] = True
    assert torch.isnan(out).all(-1).cpu().equal(hit)
    assert torch.equal(out[~hit.cuda()], want[~hit.cuda()])


@pytest.mark.parametrize("bits", [0, 2])
@pytest.mark.parametrize("flags", [1, 6])
def test_ablation_flags(kvlib, bits, flags):
    c = Cache(kvlib, 20, [150, 31], 8, 2, 32, bits, flags=flags)
    d = Drafts(c, 9)
    _check(c, d, _call(c, d))


def test_a_cache_beyond_four_gigabytes(kvlib):
    c = Cache(kvlib, 9, [300, 77], 4, 2, 64, 0, extra=70000)
    assert int(c.table.min()) * 2 * 2 * 64 * D * 2 > 1 << 32
    d = Drafts(c, 12)
    _check(c, d, _call(c, d))


@pytest.mark.parametrize("bits", [0, 2])
def test_two_graphs_at_once(kvlib, bits):
    """Captured calls with a workspace each, replayed beside one another."""
    c = Cache(kvlib, 21, [900, 400, 64], 8, 2, 32, bits)
    drafts = [Drafts(c, T, seed=T) for T in (6, 40)]
    want = [_call(c, d) for d in drafts]
    torch.cuda.synchronize()
    graphs, outs, streams, spaces = [], [], [], []   # (a graph's workspace has to outlive it)
    for d in drafts:
        st = torch.cuda.Stream()
        ws, out = c.kv.alloc_tree_workspace(c.cfg, 3, d.T, c.table.shape[1]), torch.full_like(d.q, 3.0, dtype=torch.float32)
        torch.cuda.synchronize()
        with torch.cuda.stream(st):
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=st):
                _call(c, d, ws=ws, out=out, check=False)
        graphs.append(graph), outs.append(out), streams.append(st), spaces.append(ws)
    for _ in range(5):
        for graph, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(outs, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("bits", [0, 2])
def test_a_workspace_serves_one_call_after_another(kvlib, bits):
    """A small problem behind a large one, and inputs that the kernel before wrote."""
    c = Cache(kvlib, 22, [3000, 17, 900], 8, 2, 64, bits)
    big, small = Drafts(c, 64, seed=3), Drafts(c, 64, seed=4, lens=[2, 0, 1])
    ws = c.kv.alloc_tree_workspace(c.cfg, 3, 64, c.table.shape[1])
    want = [_call(c, d) for d in (big, small)]
    for _ in range(3):
        for d, w in zip((big, small), want):
            q = d.q
            d.q = q + 0
            assert torch.equal(_call(c, d, ws=ws, check=False), w)
            d.q = q
    lens = i32([100, 17, 0])
    short = [_call(c, big, ws=x, lens=lens, check=False) for x in (ws, None)]
    assert torch.equal(*short) and c.kv.read_error(ws) == 0


@pytest.mark.parametrize("bits", [0, 2])
def test_faults_are_flagged(kvlib, bits):
    kv = kvlib
    c = Cache(kv, 23, [100, 60, 40], 8, 2, 32, bits)
    d = Drafts(c, 10, lens=[10, 4, 10])
    ws = kv.alloc_tree_workspace(c.cfg, 3, 10, c.table.shape[1])
    good = _call(c, d, ws=ws)
    for lens in ([100, -1, 40], [100, c.table.shape[1] * 32 + 1, 40]):
        out = _call(c, d, ws=ws, lens=i32(lens), check=False)
        assert kv.read_error(ws) == kv.DEVERR_POSITION
        assert torch.isnan(out[1]).all() and torch.equal(out[0], good[0]) and torch.equal(out[2], good[2])
        kv.clear_error(ws)
    for n in (-1, 11):
        d.lens = i32([10, n, 10])
        out = _call(c, d, ws=ws, check=False)
        assert kv.read_error(ws) == kv.DEVERR_POSITION
        assert torch.isnan(out[1]).all() and torch.equal(out[0], good[0]) and torch.equal(out[2], good[2])
        kv.clear_error(ws)
    d.lens = i32([10, 4, 10])
    c.table[1, 0] = c.n_pool
    out = _call(c, d, ws=ws, check=False)
    assert kv.read_error(ws) == kv.DEVERR_BLOCK_ID
    assert torch.equal(out[0], good[0]) and torch.equal(out[2], good[2])


def test_no_table_at_all(kvlib):
    """Sequences without a cached token: the drafts alone."""
    for bits in (0, 2):
        c = Cache(kvlib, 24, [0, 0], 8, 2, 32, bits)
        assert c.table.shape[1] == 0
        d = Drafts(c, 11)
        _check(c, d, _call(c, d))


@pytest.mark.parametrize("bits,B", [(0, 32), (2, 32), (3, 64), (4, 64)])
@pytest.mark.parametrize("T,n_q", [(1, 4), (5, 4), (6, 4), (7, 4), (6, 3), (7, 3), (8, 3), (9, 3), (12, 2), (13, 2), (23, 1), (24, 1), (25, 1)])
def test_few_rows(kvlib, bits, B, T, n_q):
    """Around 24 query rows a (sequence, kv head), where the packed cache's kernels change, with lengths of every kind."""
    c = Cache(kvlib, 41, [1030, 31, 0, B, 700], n_q, 1, B, bits, wild=T % 2 == 0)
    for q_dtype in (torch.float32, torch.bfloat16):
        d = Drafts(c, T, seed=T, lens=[T, T, T // 2, T, max(1, T - 1)], q_dtype=q_dtype)
        _check(c, d, _call(c, d))


@pytest.mark.parametrize("bits", [2, 4])
def test_few_rows_that_are_not_finite(kvlib, bits):
    c = Cache(kvlib, 42, [500, 33, 64], 8, 2, 32, bits)
    clean = Drafts(c, 5, lens=[5, 5, 3])
    want = _call(c, clean)
    d = Drafts(c, 5, lens=[5, 5, 3])
    d.q[2, 3:] = float("nan")
    d.q[0, 2, 3, 7] = float("nan")
    d.q[1, 1, 6, 7] = float("inf")
    out = _call(c, d)
    same = torch.ones(3, 5, 8, dtype=torch.bool, device="cuda")
    same[0, 2, 3] = same[1, 1, 6] = False
    assert torch.isnan(out[0, 2, 3]).all() and torch.isnan(out[1, 1, 6]).all()
    assert torch.equal(out[same], want[same])


@pytest.mark.parametrize("bits,q_dtype", [(0, torch.bfloat16), (0, torch.float32), (2, torch.bfloat16)])
@pytest.mark.parametrize("T", [10, 48])
def test_wait_timeout_path(kvlib, bits, q_dtype, T):
    """With the test switch the product warp of the cached tokens' kernel leaves at once: the other warps follow, the flag
    is raised, and the workspace serves the next call."""
    kv = kvlib
    c = Cache(kv, 24, [900, 400, 64], 8, 2, 64, bits)
    d = Drafts(c, T, q_dtype=q_dtype)
    ws = kv.alloc_tree_workspace(c.cfg, 3, T, c.table.shape[1])
    good = _call(c, d, ws=ws)
    c.cfg.flags |= kv.FLAG_TEST_WAIT_TIMEOUT
    for _ in range(3):
        _call(c, d, ws=ws, check=False)
        assert kv.read_error(ws) == kv.DEVERR_WAIT_TIMEOUT
        kv.clear_error(ws)
    c.cfg.flags &= ~kv.FLAG_TEST_WAIT_TIMEOUT
    assert torch.equal(_call(c, d, ws=ws), good)


@pytest.mark.parametrize("B", [32, 64])
@pytest.mark.parametrize("room", [False, True])
@pytest.mark.parametrize("T,n_q", [(33, 4), (34, 4), (35, 4), (43, 3), (45, 3), (46, 3), (65, 2), (68, 2), (69, 2)])
def test_rows_beyond_a_row_tile(kvlib, B, room, T, n_q):
    """Up to 8 query rows a (sequence, kv head) more than the 128 of one row tile, and the first counts past that; lengths
    that end anywhere in a tile, drafts that leave the rows beyond without a query, tables with room for long sequences and without."""
    c = Cache(kvlib, 43, [1030, 31, 0, 64, 700, 97, 1], n_q, 1, B, 0, wild=T % 2 == 0)
    if room:   # (columns behind the sequences are not read)
        c.table = torch.cat([c.table, torch.full((7, 50000 // B), -1, dtype=torch.int32, device="cuda")], 1).contiguous()
    for q_dtype in (torch.bfloat16, torch.float32):
        d = Drafts(c, T, seed=T, lens=[T, T, T // 2, T, T - 1, T, T], q_dtype=q_dtype)
        _check(c, d, _call(c, d))
        _check(c, d, _call(c, d, torch.bfloat16))


def test_wait_timeout_path_with_extra_rows(kvlib):
    kv = kvlib
    c = Cache(kv, 44, [900, 400, 64], 4, 1, 64, 0)
    c.table = torch.cat([c.table, torch.full((3, 2000), -1, dtype=torch.int32, device="cuda")], 1).contiguous()
    d = Drafts(c, 33)
    ws = kv.alloc_tree_workspace(c.cfg, 3, 33, c.table.shape[1])
    good = _call(c, d, ws=ws)
    c.cfg.flags |= kv.FLAG_TEST_WAIT_TIMEOUT
    for _ in range(3):
        _call(c, d, ws=ws, check=False)
        assert kv.read_error(ws) == kv.DEVERR_WAIT_TIMEOUT
        kv.clear_error(ws)
    c.cfg.flags &= ~kv.FLAG_TEST_WAIT_TIMEOUT
    assert torch.equal(_call(c, d, ws=ws), good)


def test_extra_rows_that_are_not_finite(kvlib):
    c = Cache(kvlib, 45, [300, 33, 64], 4, 1, 32, 0)
    c.table = torch.cat([c.table, torch.full((3, 4000), -1, dtype=torch.int32, device="cuda")], 1).contiguous()
    d = Drafts(c, 33, parents="chain")
    want = _call(c, d)
    d.q[0, 32, 2, 7] = float("nan")
    d.q[1, 32, 0, 9] = float("inf")
    d.q[2, 0, 1, 0] = float("nan")
    out = _call(c, d)
    same = torch.ones(3, 33, 4, dtype=torch.bool, device="cuda")
    same[0, 32, 2] = same[1, 32, 0] = same[2, 0, 1] = False
    assert torch.isnan(out[~same]).all()
    assert torch.equal(out[same], want[same])


@pytest.mark.parametrize("bits", [2, 3, 4])
@pytest.mark.parametrize("flags", [1, 6])
def test_few_rows_with_ablation_flags(kvlib, bits, flags):
    c = Cache(kvlib, 46, [150, 31], 8, 2, 32, bits, flags=flags)
    d = Drafts(c, 3)
    _check(c, d, _call(c, d))


def test_faults_with_few_rows(kvlib):
    kv = kvlib
    c = Cache(kv, 47, [100, 60, 40], 8, 2, 32, 2)
    d = Drafts(c, 4, lens=[4, 2, 4])
    ws = kv.alloc_tree_workspace(c.cfg, 3, 4, c.table.shape[1])
    good = _call(c, d, ws=ws)
    for lens in ([100, -1, 40], [100, c.table.shape[1] * 32 + 1, 40]):
        out = _call(c, d, ws=ws, lens=i32(lens), check=False)
        assert kv.read_error(ws) == kv.DEVERR_POSITION
        assert torch.isnan(out[1]).all() and torch.equal(out[0], good[0]) and torch.equal(out[2], good[2])
        kv.clear_error(ws)
    d.lens = i32([4, 5, 4])
    out = _call(c, d, ws=ws, check=False)
    assert kv.read_error(ws) == kv.DEVERR_POSITION
    assert torch.isnan(out[1]).all() and torch.equal(out[0], good[0]) and torch.equal(out[2], good[2])
    kv.clear_error(ws)
    d.lens = i32([4, 2, 4])
    c.table[1, 0] = -1
    out = _call(c, d, ws=ws, check=False)
    assert kv.read_error(ws) == kv.DEVERR_BLOCK_ID
    assert torch.equal(out[0], good[0]) and torch.equal(out[2], good[2])


def test_empty_batch(kvlib):
    kv = kvlib
    c = Cache(kv, 48, [64], 8, 2, 32, 2)
    pages = Cache(kv, 48, [64], 8, 2, 32, 0)
    q = torch.empty(0, 3, 8, D, dtype=torch.bfloat16, device="cuda")
    k = torch.empty(0, 3, 2, D, dtype=torch.bfloat16, device="cuda")
    table, lens, mask = (torch.empty(s, dtype=torch.int32, device="cuda") for s in ((0, 2), (0,), (0, 3, 1)))
    ws = kv.alloc_tree_workspace(c.cfg, 0, 3, 2)
    kv.tree_attn(c.cfg, q, c.pool, c.staging, table, lens, k, k, mask, torch.empty_like(q), ws)
    kv.tree_attn_bf16(pages.cfg, q, pages.pool, table, lens, k, k, mask, torch.empty_like(q), ws)
    assert kv.read_error(ws) == 0


@pytest.mark.parametrize("bits,B", [(2, 32), (4, 64)])
def test_few_rows_over_long_and_short_sequences(kvlib, bits, B):
    """More warps than a short sequence has blocks, and many blocks a warp."""
    c = Cache(kvlib, 49, [9000, 70, B], 4, 1, B, bits)
    for T in (1, 6):
        d = Drafts(c, T, seed=T)
        _check(c, d, _call(c, d))
