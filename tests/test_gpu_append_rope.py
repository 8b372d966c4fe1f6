"""The rotary appends against the formulas in 64 bits, and the packed one
against the bulk quantiser and the plain append.

Tolerance of a rotated value y of a pair (a, b): cos and sin are within 3e-7
(pi 2^-25 from the fp32 angle, 2 ulp of sincospif and the scale's rounding),
the product and multiply-add round twice, and a normed input is within 5e-7 of
itself (a sum of 128 squares over 4 + 5 roundings halved by the square root,
rsqrt within 2 ulp, 2 products): together below 1e-6 (|a| + |b|); a bf16
output adds half a step, 2^-8 |y|.
"""
import numpy as np
import pytest
import torch

import synth

pytestmark = pytest.mark.gpu
D = 128


def _inputs(kv, seed, counts, cached, n_q, n_kv, B, pad=0, max_blocks=None):
    g = torch.Generator().manual_seed(seed)
    cu = np.concatenate([[0], np.cumsum(counts)])
    T = int(cu[-1]) + pad
    rows = (torch.randn(T, (n_q + 2 * n_kv) * D + 8, generator=g) * 1.5).to(torch.bfloat16).cuda()
    q, k, v = (x.unflatten(1, (-1, D)) for x in (rows[:, :n_q * D], rows[:, n_q * D:(n_q + n_kv) * D],
                                                 rows[:, (n_q + n_kv) * D:(n_q + 2 * n_kv) * D]))
    nb = max_blocks or max(1, -(-int(max(c + p for c, p in zip(counts, cached))) // B))
    batch = len(counts)
    perm = np.random.default_rng(seed).permutation(batch * nb + 2).astype(np.int32)
    w = [(1 + 0.2 * torch.randn(D, generator=g)).to(torch.bfloat16).cuda() for _ in range(2)]
    i32 = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")  # noqa: E731
    return dict(q=q, k=k, v=v, cu=cu, T=T, nb=nb, n_pool=batch * nb + 2, table_np=perm[:batch * nb].reshape(batch, nb),
                table=i32(perm[:batch * nb].reshape(batch, nb)), pos=i32(cached), cu_t=i32(cu), qw=w[0], kw=w[1])


def _rope64(x, w, eps, pos, inv_freq, layout, scale):
    """(value, tolerance without output rounding) in float64: x [T][H][128], pos [T]."""
    x = x.double().cpu().numpy()
    if w is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w.double().cpu().numpy()
    r = 2 * len(inv_freq)
    ang = np.asarray(pos, np.float64)[:, None] * np.asarray(inv_freq)[None]
    c, s = (np.cos(ang) * scale)[:, None], (np.sin(ang) * scale)[:, None]
    ia, ib = (np.arange(r // 2), np.arange(r // 2) + r // 2) if layout == 0 else (np.arange(0, r, 2), np.arange(1, r, 2))
    y, tol = x.copy(), np.abs(x) * 1e-6
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    tol[..., ia] = tol[..., ib] = (np.abs(a) + np.abs(b)) * 1e-6 * max(1.0, scale)
    return y, tol


def _close(got, want, tol, dtype):
    half = torch.finfo(dtype).eps / 2
    err = np.abs(got.double().cpu().numpy() - want)
    assert np.all(err <= tol + half * np.abs(want)), float((err - tol - half * np.abs(want)).max())


CASES = [  # counts (None: decode), cached, n_q, n_kv, B, rotary, layout, norm, out dtype
    (None, [0], 1, 1, 32, 128, 0, False, torch.bfloat16),
    (None, [31, 32, 5, 1000], 8, 2, 32, 128, 0, True, torch.float32),
    (None, [63, 64, 0], 6, 3, 64, 96, 1, True, torch.bfloat16),
    (None, list(range(40)), 4, 4, 32, 64, 0, False, torch.bfloat16),
    ([1, 70, 0, 33], [0, 31, 7, 64], 8, 2, 32, 32, 0, True, torch.bfloat16),
    ([129, 1, 64, 63, 65], [0, 63, 64, 1, 63], 3, 1, 64, 16, 1, False, torch.float32),
    ([5, 0, 0, 200], [3, 0, 9, 0], 40, 10, 32, 128, 1, True, torch.bfloat16),
    ([0] * 35 + [2, 0, 3] + [1] * 40, [7] * 78, 2, 2, 64, 0, 0, True, torch.bfloat16),
    ([1100, 3], [10, 2], 4, 1, 64, 128, 0, True, torch.bfloat16),
]


@pytest.mark.parametrize("case", range(len(CASES)))
@pytest.mark.parametrize("packed", [False, True])
def test_append_rope_against_the_formulas(kvlib, case, packed):
    kv = kvlib
    counts, cached, n_q, n_kv, B, rotary, layout, norm, odt = CASES[case]
    decode = counts is None
    counts = [1] * len(cached) if decode else counts
    batch, pad = len(cached), 0 if decode else 3
    x = _inputs(kv, 10 + case, counts, cached, n_q, n_kv, B, pad)
    f, scale = kv.rope_frequencies(rotary, 10000.0, "yarn", 4.0, 512) if rotary else (np.zeros(0), 1.0)
    rope = kv.make_rope(f, layout, scale, 1e-5)
    cfg = kv.make_config(n_q, n_kv, B, 2, synth.sign_bits(3))
    ws = kv.alloc_workspace(cfg, 0, 0)
    far = torch.tensor([p + (100003 * (b % 3)) for b, p in enumerate(cached)], dtype=torch.int32, device="cuda")
    q_out = torch.full((x["T"], n_q, D), 7.0, dtype=odt, device="cuda")
    kw = dict(cu_tokens=None if decode else x["cu_t"], rope_pos=far, q_weight=x["qw"] if norm else None,
              k_weight=x["kw"] if norm else None)
    bpool = torch.full((x["n_pool"], n_kv, 2, B, D), 7.0, dtype=torch.bfloat16, device="cuda")
    kv.append_rope_bf16(cfg, rope, bpool, x["table"], x["pos"], x["q"], x["k"], x["v"], q_out, ws, **kw)
    if packed:   # keys of the bf16 append feed the bulk quantiser: the packed append's bytes are the same
        q2 = torch.full_like(q_out, 7.0)
        g = torch.Generator().manual_seed(5)
        stage = torch.randn(batch, n_kv, 2, B, D, generator=g).to(torch.bfloat16).cuda()
        before = stage.clone()
        pool = kv.alloc_pool(cfg, x["n_pool"]) + 77
        want_pool, want_stage = pool.clone(), stage.clone()
        kv.append_rope(cfg, rope, pool, stage, x["table"], x["pos"], x["q"], x["k"], x["v"], q2, ws, **kw)
        assert kv.read_error(ws) == 0
        assert torch.equal(q2, q_out)
        hb, bb = kv.head_block_bytes(cfg), kv.block_bytes(cfg)
        for b in range(batch):
            p, n = cached[b], counts[b]
            for j in range(p // B, (p + n) // B + 1):
                lo, hi = max(p, j * B), min(p + n, (j + 1) * B)
                if lo >= hi:
                    continue
                new = bpool[x["table_np"][b, j]][:, :, lo - j * B:hi - j * B]       # [n_kv][2][rows][128]
                if hi < (j + 1) * B:
                    want_stage[b, :, :, lo - j * B:hi - j * B] = new
                    continue
                rows = torch.cat([before[b, :, :, :lo - j * B], new], 2)
                for h in range(n_kv):
                    for kind in (0, 1):
                        off = torch.tensor([int(x["table_np"][b, j]) * bb + (2 * h + kind) * hb], device="cuda")
                        kv.quantize_block(cfg, kind, rows[h, kind].contiguous()[None], want_pool, ws, dst_offsets=off)
        assert torch.equal(pool, want_pool)
        assert torch.equal(stage, want_stage)
        return
    assert kv.read_error(ws) == 0
    turn = np.concatenate([[far[b].item() + i for i in range(n)] for b, n in enumerate(counts)] + [[]])
    at = np.concatenate([[cached[b] + i for i in range(n)] for b, n in enumerate(counts)] + [[]]).astype(int)
    seq = np.repeat(np.arange(batch), counts)
    n = len(at)
    want, tol = _rope64(x["q"][:n], kw["q_weight"], 1e-5, turn, f, layout, scale)
    _close(q_out[:n], want, tol, odt)
    assert torch.all(q_out[n:] == 7.0)                       # rows behind the last sequence
    want, tol = _rope64(x["k"][:n], kw["k_weight"], 1e-5, turn, f, layout, scale)
    page = torch.from_numpy(x["table_np"][seq, at // B].astype(np.int64)).cuda()
    row = torch.from_numpy(at % B).cuda()
    _close(bpool[page, :, 0, row], want, tol, torch.bfloat16)
    assert torch.equal(bpool[page, :, 1, row], x["v"][:n])
    bpool[page, :, :, row] = 7.0
    assert torch.all(bpool == 7.0)                           # nothing else was written


@pytest.mark.parametrize("B,bits", [(32, 2), (64, 3), (64, 4)])
def test_prompt_append_equals_token_by_token(kvlib, B, bits):
    """A ragged prompt, its tokens one by one, and the plain append of the rotated keys leave the same pool bytes."""
    kv = kvlib
    n_q, n_kv, counts, cached = 4, 2, [2 * B + 5, B - 3, 3 * B], [B - 2, 4, 0]
    x = _inputs(kv, B + bits, counts, cached, n_q, n_kv, B, max_blocks=5)
    cfg = kv.make_config(n_q, n_kv, B, 2, synth.sign_bits(4), bits=bits)
    rope = kv.make_rope(kv.rope_frequencies(64)[0])
    ws = kv.alloc_workspace(cfg, 0, 0)
    g = torch.Generator().manual_seed(9)
    stage0 = torch.randn(3, n_kv, 2, B, D, generator=g).to(torch.bfloat16).cuda()
    outs = []
    for way in ("prompt", "tokens", "plain"):
        pool, stage = kv.alloc_pool(cfg, x["n_pool"]), stage0.clone()
        q_out = torch.zeros_like(x["q"], memory_format=torch.contiguous_format)
        if way == "prompt":
            kv.append_rope(cfg, rope, pool, stage, x["table"], x["pos"], x["q"], x["k"], x["v"], q_out, ws,
                           cu_tokens=x["cu_t"], q_weight=x["qw"], k_weight=x["kw"])
        else:
            scratch = torch.zeros(x["n_pool"], n_kv, 2, B, D, dtype=torch.bfloat16, device="cuda")
            for i in range(max(counts)):
                on = [b for b in range(3) if i < counts[b]]
                rows = torch.tensor([int(x["cu"][b]) + i for b in on], device="cuda")
                pos = torch.tensor([cached[b] + i for b in on], dtype=torch.int32, device="cuda")
                table, st = x["table"][on].contiguous(), stage[on].contiguous()
                k, v, q = x["k"][rows], x["v"][rows], x["q"][rows]
                qo = torch.empty_like(q)
                if way == "tokens":
                    kv.append_rope(cfg, rope, pool, st, table, pos, q, k, v, qo, ws, q_weight=x["qw"], k_weight=x["kw"])
                else:
                    kv.append_rope_bf16(cfg, rope, scratch, table, pos, q, k, v, qo, ws, q_weight=x["qw"],
                                        k_weight=x["kw"])
                    page = table.long()[torch.arange(len(on)), (pos // B).long()]
                    kn = scratch[page, :, 0, (pos % B).long()].contiguous()
                    kv.append(cfg, pool, st, table, pos, kn, v.contiguous(), ws)
                stage[on] = st
                q_out[rows] = qo
        assert kv.read_error(ws) == 0
        tails = [stage[b, :, :, :(cached[b] + counts[b]) % B] for b in range(3)]
        outs.append((pool, q_out, *tails))
    for other in outs[1:]:
        for a, b in zip(outs[0], other):
            assert torch.equal(a, b)


def test_queries_in_place_without_queries_and_far_positions(kvlib):
    kv = kvlib
    cfg = kv.make_config(8, 2, 64, 2, synth.sign_bits(0))
    x = _inputs(kv, 3, [1, 1], [5, 9], 8, 2, 64)
    f = kv.rope_frequencies(128, 1e6)[0]
    rope, ws = kv.make_rope(f), kv.alloc_workspace(cfg, 0, 0)
    pool = torch.zeros(x["n_pool"], 2, 2, 64, D, dtype=torch.bfloat16, device="cuda")
    far = torch.tensor([2 ** 31 - 1, -2 ** 31], dtype=torch.int32, device="cuda")
    out = torch.empty(2, 8, D, device="cuda")
    kv.append_rope_bf16(cfg, rope, pool, x["table"], x["pos"], x["q"], x["k"], x["v"], out, ws, rope_pos=far)
    # at 2^31 the rate's two roundings leave 2^-21 rad and the oracle's product 2^-23: 6e-7 on top of the 4e-7 of
    # cosine and product for the pair of rate 1 (no norm here)
    want, tol = _rope64(x["q"], None, 0, far.cpu().numpy(), f, 0, 1.0)
    _close(out, want, 1.4 * tol, torch.float32)
    q = x["q"].contiguous()
    ref = torch.empty_like(q)
    pool2 = torch.zeros_like(pool)
    kv.append_rope_bf16(cfg, rope, pool2, x["table"], x["pos"], q, x["k"], x["v"], ref, ws, rope_pos=far)
    kv.append_rope_bf16(cfg, rope, pool2, x["table"], x["pos"], q, x["k"], x["v"], q, ws, rope_pos=far)
    assert torch.equal(q, ref) and torch.equal(pool, pool2)
    pool2.zero_()
    kv.append_rope_bf16(cfg, rope, pool2, x["table"], x["pos"], None, x["k"], x["v"], None, ws, rope_pos=far)
    assert torch.equal(pool, pool2)
    q = x["q"].contiguous()
    pk, st = kv.alloc_pool(cfg, x["n_pool"]), kv.alloc_staging(cfg, 2)
    kv.append_rope(cfg, rope, pk, st, x["table"], x["pos"], q, x["k"], x["v"], q, ws, rope_pos=far)
    assert torch.equal(q, ref) and kv.read_error(ws) == 0
    st2 = kv.alloc_staging(cfg, 2)
    kv.append_rope(cfg, rope, pk, st2, x["table"], x["pos"], None, x["k"], x["v"], None, ws, rope_pos=far)
    assert torch.equal(st, st2)


@pytest.mark.parametrize("packed", [False, True])
def test_device_faults_are_flagged_and_skip_their_sequence(kvlib, packed):
    kv = kvlib
    n_q, n_kv, B = 4, 2, 32
    cfg = kv.make_config(n_q, n_kv, B, 2, synth.sign_bits(0))
    rope, ws = kv.make_rope(kv.rope_frequencies(128)[0]), kv.alloc_workspace(cfg, 0, 0)
    x = _inputs(kv, 4, [1, 1, 1], [31, 31, 31], n_q, n_kv, B, max_blocks=2)

    def call(cu=None, pos=x["pos"], table=x["table"], T=3):
        pool = kv.alloc_pool(cfg, x["n_pool"]) if packed else torch.zeros(x["n_pool"], n_kv, 2, B, D, dtype=torch.bfloat16,
                                                                          device="cuda")
        st = kv.alloc_staging(cfg, 3)
        out = torch.zeros(T, n_q, D, device="cuda")
        a = (table, pos, x["q"][:T], x["k"][:T], x["v"][:T], out, ws)
        kv.clear_error(ws)
        if packed:
            kv.append_rope(cfg, rope, pool, st, *a, cu_tokens=cu)
        else:
            kv.append_rope_bf16(cfg, rope, pool, *a, cu_tokens=cu)
        return kv.read_error(ws), pool

    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    good, pool = call()
    assert good == 0
    for pos in ([-1, 31, 31], [31, 64, 31], [31, 31, 2 ** 31 - 1], [-2 ** 31, 31, 31]):
        err, got = call(pos=i32(pos))
        assert err == kv.DEVERR_POSITION
        for b in range(3):
            page = int(x["table_np"][b, 0])
            assert torch.equal(got[page], pool[page] if pos[b] == 31 else torch.zeros_like(pool[page]))
    for bad in (-1, x["n_pool"], -2 ** 31, 2 ** 31 - 1):
        table = x["table"].clone()
        table[1, 0] = bad
        err, got = call(table=table)
        assert err == kv.DEVERR_BLOCK_ID
        for b in (0, 2):
            page = int(x["table_np"][b, 0])
            assert torch.equal(got[page], pool[page])
    for cu in ([0, 2, 1, 3], [3, 2, 1, 0], [0, -5, 2, 3], [2 ** 31 - 1, -2 ** 31, 2 ** 31 - 1, 3]):
        err, _ = call(cu=i32(cu))
        assert err & kv.DEVERR_POSITION
    err, _ = call(cu=i32([0, 1, 2, 9]))                      # beyond the token rows
    assert err == (kv.DEVERR_POSITION if packed else 0)
    if packed:
        x["k"][1, 0, 5] = float("inf")
        err, _ = call()
        assert err == kv.DEVERR_NONFINITE


def test_offsets_past_32_bits(kvlib):
    """The last page of a pool of 2^31 elements and more, and token rows beyond 2^31 elements."""
    kv = kvlib
    cfg = kv.make_config(1, 1, 64, 2, synth.sign_bits(0))
    n_pool = (1 << 31) // (2 * 64 * D) + 3
    pool = torch.empty(n_pool, 1, 2, 64, D, dtype=torch.bfloat16, device="cuda")
    pool[-1].zero_()
    table = torch.tensor([[n_pool - 1]], dtype=torch.int32, device="cuda")
    rows = torch.empty((1 << 31) // 8 * 8 + 1024, dtype=torch.bfloat16, device="cuda")
    two = rows.as_strided((2, 1, D), (1 << 31, D, 1))
    two.copy_(torch.randn(2, 1, D))
    ws = kv.alloc_workspace(cfg, 0, 0)
    cu = torch.tensor([0, 2], dtype=torch.int32, device="cuda")
    pos = torch.tensor([3], dtype=torch.int32, device="cuda")
    rope = kv.make_rope([])
    out = torch.empty(2, 1, D, dtype=torch.bfloat16, device="cuda")
    kv.append_rope_bf16(cfg, rope, pool, table, pos, two, two, two, out, ws, cu_tokens=cu)
    assert kv.read_error(ws) == 0
    assert torch.equal(out, two) and torch.equal(pool[-1, 0, 0, 3:5], two[:, 0]) and torch.equal(pool[-1, 0, 1, 3:5], two[:, 0])
    st, pk = kv.alloc_staging(cfg, 1), kv.alloc_pool(cfg, 1)
    kv.append_rope(cfg, rope, pk, st, table, pos, two, two, two, out, ws, cu_tokens=cu)
    assert torch.equal(st[0, 0, 0, 3:5], two[:, 0])


def test_binding_refusals(kvlib):
    kv = kvlib
    cfg = kv.make_config(4, 2, 32, 2, synth.sign_bits(0))
    rope, ws = kv.make_rope([1.0] * 8), kv.alloc_workspace(cfg, 0, 0)
    x = _inputs(kv, 4, [1, 1], [0, 0], 4, 2, 32)
    pool = torch.zeros(x["n_pool"], 2, 2, 32, D, dtype=torch.bfloat16, device="cuda")
    out = torch.zeros(2, 4, D, device="cuda")
    good = dict(cfg=cfg, rope=rope, kv_pool=pool, block_table=x["table"], pos=x["pos"], q=x["q"], k=x["k"], v=x["v"],
                q_out=out, workspace=ws)
    kv.append_rope_bf16(**good)
    for bad in (dict(k=x["k"].float()), dict(k=x["k"][:1]), dict(v=x["v"].transpose(1, 2)), dict(q=x["q"][..., :64]),
                dict(q_out=out[:1]), dict(q_out=None), dict(kv_pool=pool[:, :1].contiguous()), dict(pos=x["pos"].long()),
                dict(kv_pool=pool.float()), dict(block_table=x["table"][:1]), dict(q_out=out.half()),
                dict(cu_tokens=x["cu_t"][:2]), dict(rope_pos=x["pos"][:1]), dict(q_weight=x["qw"].float()),
                dict(k_weight=x["kw"][:64]), dict(q=x["q"].cpu()), dict(workspace=ws[:128])):
        with pytest.raises(ValueError):
            kv.append_rope_bf16(**{**good, **bad})
    pk, st = kv.alloc_pool(cfg, 4), kv.alloc_staging(cfg, 2)
    good = {k: v for k, v in good.items() if k != "kv_pool"} | dict(pool=pk, staging=st)
    kv.append_rope(**good)
    for bad in (dict(staging=st[:1].contiguous()), dict(pool=pk[:, :-16].contiguous()), dict(staging=st.float())):
        with pytest.raises(ValueError):
            kv.append_rope(**{**good, **bad})


def test_captured_on_a_side_stream_equals_eager(kvlib):
    """A prompt and two decode steps captured together and replayed on another stream give the eager bytes."""
    kv = kvlib
    n_q, n_kv, B, counts, cached = 8, 2, 32, [40, 3], [20, 60]
    cfg = kv.make_config(n_q, n_kv, B, 2, synth.sign_bits(6))
    rope, ws = kv.make_rope(kv.rope_frequencies(128)[0]), kv.alloc_workspace(cfg, 0, 0)
    x = _inputs(kv, 8, counts, cached, n_q, n_kv, B, max_blocks=4)
    pool, st = kv.alloc_pool(cfg, x["n_pool"]), kv.alloc_staging(cfg, 2)
    out = torch.zeros(x["T"], n_q, D, dtype=torch.bfloat16, device="cuda")
    steps = [x["pos"] + torch.tensor(counts, dtype=torch.int32, device="cuda") + i for i in range(2)]

    def work():
        kv.append_rope(cfg, rope, pool, st, x["table"], x["pos"], x["q"], x["k"], x["v"], out, ws, cu_tokens=x["cu_t"])
        for p in steps:
            kv.append_rope(cfg, rope, pool, st, x["table"], p, None, x["k"][:2], x["v"][:2], None, ws)

    work()
    torch.cuda.synchronize()
    want = pool.clone(), st.clone(), out.clone()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=side):
        work()
    for _ in range(2):
        for t in (pool, st, out):
            t.zero_()
        st.copy_(torch.zeros_like(st))
        # the first block takes staged rows: give it the same ones as the eager run had (zeros)
        with torch.cuda.stream(side):
            side.wait_stream(torch.cuda.default_stream())
            graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(pool, want[0]) and torch.equal(st, want[1]) and torch.equal(out, want[2])
    assert kv.read_error(ws) == 0
