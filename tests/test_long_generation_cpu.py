"""Drafted trees, kept weights and eviction without a GPU: the mask of a tree, the
refusals of the C entry points."""
import ctypes

import numpy as np
import pytest
import torch

import bit_kv_cache_08_gb300 as kv
import synth

INV, WS = -1, -4


@pytest.fixture(scope="module", autouse=True)
def built():
    kv.build()


def _cfg(**more):
    base = dict(n_q_heads=8, n_kv_heads=2, block_size=32, varn_iters=2, sign_bits=synth.sign_bits(1))
    base.update(more)
    return kv.make_config(**base)


def _bits(mask, T):
    w = mask.numpy().view(np.uint32)
    return (w[..., None] >> np.arange(32, dtype=np.uint32) & 1).astype(bool).reshape(*w.shape[:-1], -1)[..., :T]


@pytest.mark.parametrize("T", [1, 2, 31, 32, 33, 64, 100, 128])
def test_tree_mask_shows_ancestors_and_oneself(T):
    r = np.random.default_rng(T)
    parents = np.stack([[int(r.integers(-1, i)) if i else -1 for i in range(T)] for _ in range(3)])
    mask = kv.tree_mask(parents)
    assert mask.dtype is torch.int32 and tuple(mask.shape) == (3, T, (T + 31) // 32)
    shown = _bits(mask, T)
    for b in range(3):
        for i in range(T):
            want, j = set(), i
            while j >= 0:
                want.add(j)
                j = parents[b, j]
            assert set(np.nonzero(shown[b, i])[0]) == want
    assert torch.equal(kv.tree_mask(parents[1]), mask[1])
    assert torch.equal(kv.tree_mask(parents[1].tolist()), mask[1])


@pytest.mark.parametrize("parents", [[], [0], [-2], [-1, 1], [-1, 2, 0], [0.5], [[[-1]]], [-1] * 129])
def test_tree_mask_refuses(parents):
    with pytest.raises(ValueError):
        kv.tree_mask(parents)


def test_workspace_queries_refuse_bad_sizes():
    c = _cfg()
    for args in ((-1, 4, 4), (2, 0, 4), (2, 129, 4), (2, 4, -1), (1 << 27, 128, 4), (2, 4, 1 << 27)):
        assert kv.tree_workspace_bytes(c, *args) == 0, args
    for args in ((-1, 4), (2, -1), (1 << 30, 4), (2, 1 << 27)):
        assert kv.weights_workspace_bytes(c, *args) == 0, args
    bad = _cfg(bits=5)
    assert kv.tree_workspace_bytes(bad, 2, 4, 4) == 0 and kv.weights_workspace_bytes(bad, 2, 4) == 0
    assert kv.tree_workspace_bytes(c, 0, 4, 4) >= 256 and kv.weights_workspace_bytes(c, 0, 4) >= 256


P, ODD = 1 << 20, (1 << 20) + 2   # pointers that are never followed


def _tree(bf16, **more):
    a = dict(cfg=_cfg(), q=P, qd=0, pool=P, n=4, staging=P, table=P, blocks=4, lens=P, k=P, v=P, ks=256, vs=256, mask=P,
             drafts_of=None, batch=2, drafts=4, out=P, od=0, ws=P, wsn=1 << 40)
    a.update(more)
    head = (ctypes.byref(a["cfg"]), a["q"], a["qd"], a["pool"], a["n"])
    rest = (a["table"], a["blocks"], a["lens"], a["k"], a["v"], a["ks"], a["vs"], a["mask"], a["drafts_of"], a["batch"],
            a["drafts"], a["out"], a["od"], a["ws"], a["wsn"], None)
    L = kv.lib()
    return L.kvarn_tree_attn_bf16(*head, *rest) if bf16 else L.kvarn_tree_attn(*head, a["staging"], *rest)


@pytest.mark.parametrize("bf16", [False, True])
def test_tree_attention_refuses(bf16):
    for more in (dict(q=None), dict(q=ODD), dict(qd=2), dict(od=2), dict(pool=None), dict(pool=ODD), dict(n=0), dict(table=None),
                 dict(table=P + 1), dict(blocks=-1), dict(blocks=1 << 27), dict(lens=None), dict(k=None), dict(k=ODD), dict(v=None),
                 dict(v=ODD), dict(ks=252), dict(ks=128), dict(vs=260), dict(vs=0), dict(mask=None), dict(mask=P + 2),
                 dict(drafts_of=P + 2), dict(batch=-1), dict(drafts=0), dict(drafts=129), dict(out=None), dict(out=ODD),
                 dict(ws=None), dict(ws=P + 8), dict(batch=1 << 28, drafts=128), dict(batch=1 << 20)):
        assert _tree(bf16, **more) == INV, more
    if not bf16:
        assert _tree(bf16, staging=None) == INV and _tree(bf16, staging=ODD) == INV
    assert _tree(bf16, cfg=_cfg(n_q_heads=7)) == INV and _tree(bf16, cfg=_cfg(bits=5)) == -2
    assert _tree(bf16, batch=0) == 0


def _weights(bf16, **more):
    a = dict(cfg=_cfg(), q=P, qd=0, pool=P, n=4, staging=P, table=P, blocks=4, lens=P, batch=2, out=P, od=0, win=P, wout=P,
             stride=128, decay=1.0, ws=P, wsn=1 << 40)
    a.update(more)
    head = (ctypes.byref(a["cfg"]), a["q"], a["qd"], a["pool"], a["n"])
    rest = (a["table"], a["blocks"], a["lens"], a["batch"], a["out"], a["od"], a["win"], a["wout"], a["stride"], a["decay"],
            a["ws"], a["wsn"], None)
    L = kv.lib()
    return L.kvarn_decode_attn_weights_bf16(*head, *rest) if bf16 else L.kvarn_decode_attn_weights(*head, a["staging"], *rest)


@pytest.mark.parametrize("bf16", [False, True])
def test_decode_attention_with_weights_refuses(bf16):
    for more in (dict(q=None), dict(qd=3), dict(od=-1), dict(pool=ODD), dict(n=0), dict(table=None), dict(blocks=-1), dict(lens=None),
                 dict(batch=-1), dict(out=None), dict(out=ODD), dict(win=P + 4), dict(wout=None), dict(wout=P + 8), dict(stride=124),
                 dict(stride=130), dict(stride=-4), dict(decay=-0.1), dict(decay=1.5), dict(decay=float("nan")), dict(ws=None),
                 dict(ws=P + 8)):
        assert _weights(bf16, **more) == INV, more
    assert _weights(bf16, batch=0) == 0


def _evict(bf16, **more):
    a = dict(cfg=_cfg(), pool=P, n=4, table=P, blocks=4, lens=P, w=P, stride=128, budget=64, recent=32, new_table=P, new_blocks=3,
             new_lens=2 * P, new_w=2 * P, new_stride=96, kept=P, batch=2, ws=P)
    a.update(more)
    f = kv.lib().kvarn_evict_bf16 if bf16 else kv.lib().kvarn_evict
    return f(ctypes.byref(a["cfg"]), a["pool"], a["n"], a["table"], a["blocks"], a["lens"], a["w"], a["stride"], a["budget"],
             a["recent"], a["new_table"], a["new_blocks"], a["new_lens"], a["new_w"], a["new_stride"], a["kept"], a["batch"],
             a["ws"], None)


@pytest.mark.parametrize("bf16", [False, True])
def test_eviction_refuses(bf16):
    for more in (dict(pool=None), dict(pool=ODD), dict(n=0), dict(n=1 << 31), dict(table=None), dict(blocks=-1), dict(blocks=1 << 27),
                 dict(lens=None), dict(w=None), dict(w=P + 8), dict(stride=124), dict(stride=130), dict(budget=0), dict(budget=-32),
                 dict(recent=-32), dict(recent=96), dict(new_table=None), dict(new_blocks=1), dict(new_blocks=-1),
                 dict(new_lens=None), dict(new_lens=P), dict(new_w=None), dict(new_w=P), dict(new_stride=95), dict(kept=None),
                 dict(kept=P + 2), dict(batch=-1), dict(ws=None), dict(ws=P + 8)):
        assert _evict(bf16, **more) == INV, more
    if not bf16:   # whole blocks, and room for the tail
        assert _evict(bf16, budget=65) == INV and _evict(bf16, recent=31) == INV and _evict(bf16, new_blocks=2, new_stride=64) == INV
    assert _evict(bf16, batch=0) == 0
