"""A generation that uses the tree, the kept weights and the eviction together over
one cache, and the refusals of their binding."""
import numpy as np
import pytest
import torch

from cache_util import Cache, attend, close_rows, i32

pytestmark = pytest.mark.gpu
D = 128


@pytest.mark.parametrize("bits", [0, 2])
def test_drafts_weights_and_eviction_over_one_cache(kvlib, bits):
    """Prompt; then rounds of: a drafted chain verified, its accepted part appended, decode steps that keep
    their weights, and an eviction. Every output is held against the cache's own bytes in 64 bits."""
    kv = kvlib
    B, n_q, n_kv, T, budget, recent = 32, 8, 2, 9, 96, 32
    G = n_q // n_kv
    lens = [150, 70, 31]
    batch, blocks = len(lens), 8
    c = Cache(kv, 50, lens, n_q, n_kv, B, bits, blocks=blocks, spare=2 * batch * blocks)
    pages = c.spare_np.reshape(2, batch, blocks)
    g = torch.Generator(device="cuda").manual_seed(3)
    rope = kv.make_rope([])
    ws, tree_ws = kv.alloc_weights_workspace(c.cfg, batch, blocks), kv.alloc_tree_workspace(c.cfg, batch, T, blocks)
    weights = torch.zeros(batch, n_kv, blocks * B, device="cuda")
    expect = np.zeros((batch, n_kv, blocks * B))
    slack = np.zeros_like(expect)
    mask = kv.tree_mask([list(range(-1, T - 1))] * batch).cuda()

    def append(k, v, counts):
        cu = i32(np.concatenate([[0], np.cumsum(counts)]))
        if bits:
            kv.append_rope(c.cfg, rope, c.pool, c.staging, c.table, c.seq_lens, None, k, v, None, ws, cu_tokens=cu)
        else:
            kv.append_rope_bf16(c.cfg, rope, c.pool, c.table, c.seq_lens, None, k, v, None, ws, cu_tokens=cu)
        c.seq_lens = c.seq_lens + i32(counts)
        c.lens = c.seq_lens.tolist()

    for turn in range(2):
        # ---- drafts
        q = torch.randn(batch, T, n_q, D, generator=g, device="cuda").to(torch.bfloat16)
        k, v = (torch.randn(batch, T, n_kv, D, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
        out = torch.zeros(batch, T, n_q, D, dtype=torch.bfloat16, device="cuda")
        if bits:
            kv.tree_attn(c.cfg, q, c.pool, c.staging, c.table, c.seq_lens, k, v, mask, out, tree_ws)
        else:
            kv.tree_attn_bf16(c.cfg, q, c.pool, c.table, c.seq_lens, k, v, mask, out, tree_ws)
        for b in range(batch):
            for h in range(n_kv):
                (K, V), (ek, ev) = c.tokens(b, h)
                kb, vb, qb, ob = (x[b].double().cpu().numpy() for x in (k, v, q, out))
                K, V = np.concatenate([K, kb[:, h]]), np.concatenate([V, vb[:, h]])
                ek, ev = np.concatenate([ek, np.linalg.norm(kb[:, h], axis=1)]), np.concatenate([ev, np.linalg.norm(vb[:, h], axis=1)])
                see = np.concatenate([np.ones((T, c.lens[b]), bool), np.tri(T, dtype=bool)], 1).repeat(G, 0)
                want, tol, _, _ = attend(qb[:, h * G:(h + 1) * G].reshape(-1, D), K, V, ek, ev, c.scale, False, see)
                close_rows(ob[:, h * G:(h + 1) * G].reshape(-1, D), want, tol, True)
        # ---- the accepted ones, a different number a sequence
        counts = [3 + turn, 0, T]
        append(torch.cat([k[b, :n] for b, n in enumerate(counts)]), torch.cat([v[b, :n] for b, n in enumerate(counts)]), counts)
        # ---- decode steps
        for _ in range(3):
            q1 = torch.randn(batch, n_q, D, generator=g, device="cuda").to(torch.bfloat16)
            k1, v1 = (torch.randn(batch, n_kv, D, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
            append(k1, v1, [1] * batch)
            out1 = torch.zeros(batch, n_q, D, device="cuda")
            if bits:
                kv.decode_attn_weights(c.cfg, q1, c.pool, c.staging, c.table, c.seq_lens, out1, weights, ws)
            else:
                kv.decode_attn_weights_bf16(c.cfg, q1, c.pool, c.table, c.seq_lens, out1, weights, ws)
            for b in range(batch):
                for h in range(n_kv):
                    (K, V), (ek, ev) = c.tokens(b, h)
                    qb, ob = (x[b, h * G:(h + 1) * G].double().cpu().numpy() for x in (q1, out1))
                    want, tol, p, off = attend(qb, K, V, ek, ev, c.scale, False)
                    close_rows(ob, want, tol, False)
                    expect[b, h, :c.lens[b]] += p.sum(0)
                    slack[b, h, :c.lens[b]] += off.sum(0) + 6 * 2.0 ** -24 * expect[b, h, :c.lens[b]]
        got = weights.double().cpu().numpy()
        assert (np.abs(got - expect) <= slack).all()
        # ---- eviction to fresh pages
        new_table = torch.from_numpy(pages[turn]).cuda()
        new_lens, new_weights = torch.zeros_like(c.seq_lens), torch.zeros_like(weights)
        kept = torch.zeros(batch, n_kv, budget // B if bits else budget, dtype=torch.int32, device="cuda")
        before = [[c.tokens(b, h) for h in range(n_kv)] for b in range(batch)]
        (kv.evict if bits else kv.evict_bf16)(c.cfg, c.pool, c.table, c.seq_lens, weights, new_table, new_lens, new_weights, kept,
                                              ws, budget=budget, recent=recent)
        old = c.lens
        c.table, c.table_np, c.seq_lens, c.lens, weights = new_table, pages[turn], new_lens, new_lens.tolist(), new_weights
        unit = B if bits else 1
        for b in range(batch):
            assert c.lens[b] == min(old[b] - old[b] % unit, budget) + old[b] % unit
            for h in range(n_kv):
                at = kept[b, h].cpu().numpy()
                at = at[at >= 0]
                at = np.concatenate([(at[:, None] * unit + np.arange(unit)).ravel(), np.arange(old[b] - old[b] % unit, old[b])])
                (K, V), _ = c.tokens(b, h)
                assert (K == before[b][h][0][0][at]).all() and (V == before[b][h][0][1][at]).all()
                moved, moved_slack = expect[b, h, at], slack[b, h, at]
                expect[b, h], slack[b, h] = 0.0, 0.0
                expect[b, h, :len(at)], slack[b, h, :len(at)] = moved, moved_slack
        assert kv.read_error(ws) == 0 and kv.read_error(tree_ws) == 0


def _tree(kv, **more):
    cfg = kv.make_config(8, 2, 32, 2, [0] * 4)
    z = lambda *s, dtype=torch.bfloat16: torch.zeros(*s, dtype=dtype, device="cuda")  # noqa: E731
    a = dict(q=z(2, 4, 8, D), pool=z(6, 2, 2, 32, D), table=z(2, 3, dtype=torch.int32), lens=z(2, dtype=torch.int32),
             k=z(2, 4, 2, D), v=z(2, 4, 2, D), mask=z(2, 4, 1, dtype=torch.int32), out=z(2, 4, 8, D),
             ws=kv.alloc_tree_workspace(cfg, 2, 4, 3), draft_lens=None)
    a.update(more)
    kv.tree_attn_bf16(cfg, a["q"], a["pool"], a["table"], a["lens"], a["k"], a["v"], a["mask"], a["out"], a["ws"],
                      draft_lens=a["draft_lens"])


def test_the_tree_binding_refuses(kvlib):
    z = lambda *s, dtype=torch.bfloat16: torch.zeros(*s, dtype=dtype, device="cuda")  # noqa: E731
    i = torch.int32
    _tree(kvlib)
    _tree(kvlib, q=z(2, 4, 8, D, dtype=torch.float32), out=z(2, 4, 8, D, dtype=torch.float32), draft_lens=z(2, dtype=i))
    for more in (dict(q=z(2, 4, 8, D).cpu()), dict(q=z(2, 4, 6, D)), dict(q=z(2, 5, 8, D)), dict(q=z(2, 4, 8, D, dtype=torch.float16)),
                 dict(q=z(2, 8, 4, D).transpose(1, 2)), dict(pool=z(6, 2, 2, 64, D)), dict(pool=z(6, 2, 2, 32, D).float()),
                 dict(table=z(3, 3, dtype=i)), dict(table=z(2, 3, dtype=torch.int64)), dict(table=z(3, 2, dtype=i).T), dict(lens=z(3, dtype=i)),
                 dict(k=z(2, 4, 4, D)), dict(k=z(2, 4, 2, D).float()), dict(v=z(2, 2, 4, D).transpose(1, 2)), dict(v=z(2, 8, 2, D)[:, :4]),
                 dict(mask=z(2, 4, 2, dtype=i)), dict(mask=z(2, 4, 1, dtype=torch.int64)), dict(out=z(2, 4, 8, D, dtype=torch.float16)),
                 dict(out=z(2, 4, 2, D)), dict(ws=z(64, dtype=i)), dict(draft_lens=z(3, dtype=i)), dict(draft_lens=z(2)), dict(k=None)):
        with pytest.raises(ValueError):
            _tree(kvlib, **more)
    with pytest.raises(kvlib.KVarNError) as e:
        _tree(kvlib, ws=z(16, dtype=torch.uint8))
    assert e.value.status == -4


def test_the_weights_binding_refuses(kvlib):
    kv = kvlib
    cfg = kv.make_config(8, 2, 32, 2, [0] * 4)
    z = lambda *s, dtype=torch.float32: torch.zeros(*s, dtype=dtype, device="cuda")  # noqa: E731
    i = torch.int32

    def call(**more):
        a = dict(q=z(2, 8, D), pool=z(6, 2, 2, 32, D, dtype=torch.bfloat16), table=z(2, 3, dtype=i), lens=z(2, dtype=i), out=z(2, 8, D),
                 w=z(2, 2, 96), w_in=None, ws=kv.alloc_weights_workspace(cfg, 2, 3), decay=1.0)
        a.update(more)
        kv.decode_attn_weights_bf16(cfg, a["q"], a["pool"], a["table"], a["lens"], a["out"], a["w"], a["ws"], weights_in=a["w_in"],
                                    decay=a["decay"])

    call()
    call(w=z(2, 2, 100), w_in=z(2, 2, 100), decay=0.5)
    for more in (dict(q=z(2, 6, D)), dict(out=z(2, 8, D, dtype=torch.float16)), dict(w=z(2, 1, 96)), dict(w=z(2, 2, 96, dtype=torch.bfloat16)),
                 dict(w=z(2, 2, 96).cpu()), dict(w_in=z(2, 2, 100)), dict(w_in=z(2, 2, 96, dtype=torch.float64)), dict(w=z(2, 96, 2).transpose(1, 2)),
                 dict(lens=z(1, dtype=i)), dict(table=z(1, 3, dtype=i)), dict(ws=z(256))):
        with pytest.raises(ValueError):
            call(**more)
    for more in (dict(w=z(2, 2, 92)), dict(w=z(2, 2, 98)), dict(decay=2.0), dict(ws=z(300, dtype=torch.uint8))):
        with pytest.raises(kv.KVarNError):
            call(**more)


@pytest.mark.parametrize("bits", [0, 2])
def test_the_evict_binding_refuses(kvlib, bits):
    kv = kvlib
    cfg = kv.make_config(2, 2, 32, 2, [0] * 4)
    z = lambda *s, dtype=torch.int32: torch.zeros(*s, dtype=dtype, device="cuda")  # noqa: E731
    f = torch.float32
    pool = kv.alloc_pool(cfg, 12) if bits else z(12, 2, 2, 32, D, dtype=torch.bfloat16)

    def call(**more):
        a = dict(pool=pool, table=z(2, 4), lens=z(2), w=z(2, 2, 128, dtype=f), new_table=z(2, 3) + 4, new_lens=z(2), new_w=z(2, 2, 96, dtype=f),
                 kept=z(2, 2, 2 if bits else 64), ws=kv.alloc_workspace(cfg, 0, 0), budget=64, recent=32)
        a.update(more)
        (kv.evict if bits else kv.evict_bf16)(cfg, a["pool"], a["table"], a["lens"], a["w"], a["new_table"], a["new_lens"], a["new_w"],
                                              a["kept"], a["ws"], budget=a["budget"], recent=a["recent"])

    call()
    for more in (dict(pool=pool.cpu()), dict(pool=pool.flatten()), dict(table=z(3, 4)), dict(lens=z(2, dtype=f)), dict(w=z(2, 1, 128, dtype=f)),
                 dict(w=z(2, 2, 128)), dict(new_table=z(1, 3)), dict(new_lens=z(3)), dict(new_w=z(2, 2, 96)), dict(new_w=z(96, 2, 2, dtype=f)),
                 dict(kept=z(2, 2, 5)), dict(kept=z(2, 2, 64, dtype=torch.int64)), dict(ws=z(100, dtype=torch.uint8)), dict(table=None)):
        with pytest.raises(ValueError):
            call(**more)
    lens = z(2)
    for more in (dict(recent=96), dict(recent=-32), dict(w=z(2, 2, 124, dtype=f)), dict(new_w=z(2, 2, 64, dtype=f)), dict(lens=lens, new_lens=lens)):
        with pytest.raises(kv.KVarNError):
            call(**more)
