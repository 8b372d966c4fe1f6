"""Decode attention that keeps its weights, against softmax in 64 bits over the same
cache bytes (tolerances: cache_util) and against the decode attention it extends."""
import numpy as np
import pytest
import torch

from cache_util import Cache, attend, close_rows, i32

pytestmark = pytest.mark.gpu
D = 128


def _call(c, q, weights, out_dtype=torch.float32, weights_in=None, decay=1.0, ws=None, lens=None, out=None, check=True):
    kv = c.kv
    out = torch.full(q.shape, 3.0, dtype=out_dtype, device="cuda") if out is None else out
    ws = kv.alloc_weights_workspace(c.cfg, q.shape[0], c.table.shape[1]) if ws is None else ws
    lens = c.seq_lens if lens is None else lens
    if c.bits:
        kv.decode_attn_weights(c.cfg, q, c.pool, c.staging, c.table, lens, out, weights, ws, weights_in=weights_in, decay=decay)
    else:
        kv.decode_attn_weights_bf16(c.cfg, q, c.pool, c.table, lens, out, weights, ws, weights_in=weights_in, decay=decay)
    if check:
        assert kv.read_error(ws) == 0
    return out


def _decode(c, q):
    kv = c.kv
    out = torch.full(q.shape, 3.0, device="cuda")
    ws = kv.alloc_workspace(c.cfg, q.shape[0], c.table.shape[1])
    if c.bits:
        kv.decode_attn(c.cfg, q, c.pool, c.staging, c.table, c.seq_lens, out, ws)
    else:
        kv.decode_attn_bf16(c.cfg, q, c.pool, c.table, c.seq_lens, out, ws)
    return out


def _check(c, q, out, got, before, decay, seqs=None):
    n_q, n_kv = c.cfg.n_q_heads, c.n_kv
    G = n_q // n_kv
    qn, on, gn, bn = (x.double().cpu().numpy() for x in (q, out, got, before))
    for b in range(len(c.lens)) if seqs is None else seqs:
        L = c.lens[b]
        for h in range(n_kv):
            (K, V), (ek, ev) = c.tokens(b, h)
            rows = slice(h * G, (h + 1) * G)
            want, tol, p, off = attend(qn[b, rows], K, V, ek, ev, c.scale, q.dtype is torch.float32)
            close_rows(on[b, rows], want, tol, out.dtype is torch.bfloat16)
            new = decay * bn[b, h, :L] + p.sum(0)
            # the sum of 1 + G terms rounds at each of them; a term below 2^-126, fp32's least normal
            # number, may become 0 or that number
            over = np.abs(gn[b, h, :L] - new) - (off.sum(0) + 6 * 2.0 ** -24 * new + G * 2.0 ** -126)
            assert over.max(initial=-1.0) <= 0, f"sequence {b} head {h}: {over.max()} beyond the bound"
            assert (gn[b, h, L:] == 7.0).all(), "behind the end"


@pytest.mark.parametrize("bits,B,n_q,n_kv", [(0, 32, 8, 2), (0, 64, 3, 1), (2, 32, 8, 2), (2, 64, 6, 2), (3, 64, 4, 4),
                                             (3, 32, 12, 4), (4, 64, 8, 2), (4, 32, 2, 1)])
@pytest.mark.parametrize("q_dtype", [torch.bfloat16, torch.float32])
def test_against_64_bits(kvlib, bits, B, n_q, n_kv, q_dtype):
    lens = [0, 1, B - 1, B, B + 1, 5 * B + 7, 313, 2]
    c = Cache(kvlib, 11 + bits, lens, n_q, n_kv, B, bits)
    g = torch.Generator(device="cuda").manual_seed(5)
    q = (2 * torch.randn(len(lens), n_q, D, generator=g, device="cuda")).to(q_dtype)
    cols = c.table.shape[1] * B + 4
    before = torch.rand(len(lens), n_kv, cols, generator=g, device="cuda") * 3
    got = torch.full_like(before, 7.0)
    out = _call(c, q, got, weights_in=before, decay=0.75)
    _check(c, q, out, got, before, 0.75)
    # the output is the decode attention's, bit for bit
    assert torch.equal(out, _decode(c, q))
    # bf16 output: the same values rounded once
    half = _call(c, q, torch.zeros_like(before), torch.bfloat16)
    assert torch.equal(half, out.to(torch.bfloat16))


@pytest.mark.parametrize("bits", [0, 2])
@pytest.mark.parametrize("batch,ctx", [(1, 20000), (40, 700), (150, 90)])
def test_few_long_and_many_short_sequences(kvlib, bits, batch, ctx):
    """Both merges, with their raw tail rows, and units of many chunks of the weights' kernel."""
    lens = np.random.default_rng(batch).integers(ctx // 2, ctx + 1, batch)
    c = Cache(kvlib, 3, lens, 8, 2, 64, bits, wild=batch == 40)
    q = torch.randn(batch, 8, D, device="cuda").to(torch.bfloat16)
    before = torch.zeros(batch, 2, c.table.shape[1] * 64, device="cuda")
    got = torch.full_like(before, 7.0)
    out = _call(c, q, got, weights_in=before)
    _check(c, q, out, got, before, 1.0, range(0, batch, 1 + batch // 6))


@pytest.mark.parametrize("bits", [0, 2])
def test_accumulates_in_place_from_step_to_step(kvlib, bits):
    c = Cache(kvlib, 4, [70, 0, 129], 4, 2, 32, bits)
    ws = c.kv.alloc_weights_workspace(c.cfg, 3, c.table.shape[1])
    q = [torch.randn(3, 4, D, device="cuda") for _ in range(3)]
    total = torch.zeros(3, 2, c.table.shape[1] * 32, device="cuda")
    steps = []
    for x in q:
        one = torch.zeros_like(total)
        _call(c, x, one, ws=ws, decay=0.0)
        steps.append(one)
    for x in q:
        _call(c, x, total, ws=ws, decay=0.5)
    want = ((steps[0].double() * 0.5 + steps[1].double()) * 0.5 + steps[2].double())
    assert (total.double() - want).abs().max() <= 4 * 2.0 ** -24 * 4    # two roundings a step of values below 4
    # each row of weights sums to its query heads, where there is a token
    sums = steps[0].double().sum(-1).cpu()
    assert torch.allclose(sums, torch.tensor([[2.0, 2.0], [0.0, 0.0], [2.0, 2.0]], dtype=torch.float64), atol=2 * 2.0 ** -15)


@pytest.mark.parametrize("bits", [0, 2])
def test_earlier_weights_are_not_read_without_decay(kvlib, bits):
    c = Cache(kvlib, 6, [50, 64], 4, 2, 32, bits)
    q = torch.randn(2, 4, D, device="cuda").to(torch.bfloat16)
    got = torch.full((2, 2, c.table.shape[1] * 32), float("nan"), device="cuda")
    _call(c, q, got, decay=0.0)
    assert torch.isfinite(got[0, :, :50]).all() and torch.isnan(got[0, :, 50:]).all() and torch.isfinite(got[1]).all()


@pytest.mark.parametrize("bits", [0, 2])
def test_graph_replay_on_another_stream(kvlib, bits):
    c = Cache(kvlib, 8, [200, 33, 64], 8, 2, 32, bits)
    q = torch.randn(3, 8, D, device="cuda").to(torch.bfloat16)
    before = torch.rand(3, 2, c.table.shape[1] * 32, device="cuda")
    eager = torch.full_like(before, 7.0)
    out = _call(c, q, eager, weights_in=before)
    ws = c.kv.alloc_weights_workspace(c.cfg, 3, c.table.shape[1])
    got, out2, w2 = torch.full_like(before, 7.0), torch.zeros_like(out), before.clone()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            _call(c, q, got, weights_in=w2, ws=ws, out=out2, check=False)
        for _ in range(3):
            graph.replay()
    side.synchronize()
    assert torch.equal(got, eager) and torch.equal(out, out2)


def test_a_cache_beyond_four_gigabytes(kvlib):
    """Blocks whose byte offsets do not fit 32 bits."""
    c = Cache(kvlib, 9, [300, 77], 4, 2, 64, 0, extra=70000)
    assert int(c.table.min()) * 2 * 2 * 64 * D * 2 > 1 << 32
    q = torch.randn(2, 4, D, device="cuda").to(torch.bfloat16)
    before = torch.zeros(2, 2, c.table.shape[1] * 64, device="cuda")
    got = torch.full_like(before, 7.0)
    out = _call(c, q, got, weights_in=before)
    _check(c, q, out, got, before, 1.0)


@pytest.mark.parametrize("bits", [0, 2])
def test_faults_are_flagged(kvlib, bits):
    kv = kvlib
    c = Cache(kv, 10, [100, 60, 40], 4, 2, 32, bits)
    q = torch.randn(3, 4, D, device="cuda").to(torch.bfloat16)
    ws = kv.alloc_weights_workspace(c.cfg, 3, c.table.shape[1])
    good = torch.full((3, 2, c.table.shape[1] * 32), 7.0, device="cuda")
    _call(c, q, good, decay=0.0, ws=ws)
    got = torch.full_like(good, 7.0)
    _call(c, q, got, decay=0.0, ws=ws, lens=i32([100, -1, 40]), check=False)
    assert kv.read_error(ws) == kv.DEVERR_POSITION
    assert torch.equal(got[0], good[0]) and torch.equal(got[2], good[2]) and (got[1] == 7.0).all()
    kv.clear_error(ws)
    _call(c, q, got, decay=0.0, ws=ws, lens=i32([100, c.table.shape[1] * 32 + 1, 40]), check=False)
    assert kv.read_error(ws) == kv.DEVERR_POSITION and (got[1] == 7.0).all()
    kv.clear_error(ws)
    c.table[1, 0] = c.n_pool
    _call(c, q, got, decay=0.0, ws=ws, check=False)
    assert kv.read_error(ws) & kv.DEVERR_BLOCK_ID
    assert torch.equal(got[0], good[0]) and torch.equal(got[2], good[2])
