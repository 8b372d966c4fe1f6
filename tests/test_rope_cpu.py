"""Rotary positions on the host: the fixed-point rates, the frequency
scalings, and the argument checks of the rotary appends (nothing is launched)."""
import ctypes
import math
from fractions import Fraction

import numpy as np
import pytest

import bit_kv_cache_08_gb300 as kv
import synth

INV, UNS = -1, -2


@pytest.fixture(scope="module", autouse=True)
def built():
    kv.build()


# pi to 60 digits
PI = Fraction(3141592653589793238462643383279502884197169399375105820974944, 10 ** 60)


@pytest.mark.parametrize("rotary,theta", [(128, 10000.0), (96, 1e6), (16, 5e5)])
def test_rates_are_turns_per_position(rotary, theta):
    """Each rate is within 2^-53 of itself (two roundings to 53 bits: the constant's and the product's) plus 2^-65."""
    f = theta ** (-np.arange(0, rotary, 2) / rotary)
    r = kv.make_rope(f, layout=kv.ROPE_INTERLEAVED, scale=0.5, eps=1e-5)
    assert r.rotary_dim == rotary and r.layout == kv.ROPE_INTERLEAVED and r.scale == 0.5
    for i, x in enumerate(f):
        want = Fraction(float(x)) / (2 * PI)
        got = Fraction(r.turns[i], 1 << 64)
        assert abs(got - want) <= want / (1 << 52) + Fraction(1, 1 << 65)


def test_rates_of_whole_turns_and_negative_rates():
    r = kv.make_rope([0.0, 2 * math.pi * 0.25, -2 * math.pi * 0.25, 2 * math.pi * 7.5, 0, 0, 0, 0])
    q = 1 << 62
    for i, want in ((0, 0), (1, q), (2, 3 * q), (3, 2 * q)):
        d = (r.turns[i] - want) % (1 << 64)
        assert min(d, (1 << 64) - d) <= 1 << 14      # 7.5 turns: an ulp of 8 is 2^-50 turns


def test_frequency_scalings():
    base, one = kv.rope_frequencies(64, 10000.0)
    assert one == 1.0 and base[0] == 1.0 and np.isclose(base[-1], 10000.0 ** (-62 / 64), rtol=1e-14)
    lin, _ = kv.rope_frequencies(64, 10000.0, "linear", 4.0)
    assert np.allclose(lin, base / 4, rtol=1e-15)
    ntk, _ = kv.rope_frequencies(64, 10000.0, "ntk", 4.0)
    assert ntk[0] == 1.0 and np.isclose(ntk[-1], base[-1] / 4, rtol=1e-12)
    for kind, scale in (("bands", 1.0), ("yarn", 0.1 * math.log(8.0) + 1)):
        f, s = kv.rope_frequencies(64, 10000.0, kind, 8.0, original_ctx=4096, low=1.0, high=4.0)
        assert np.isclose(s, scale, rtol=1e-15)
        turns = 4096 * base / (2 * np.pi)
        assert np.allclose(f[turns >= 4], base[turns >= 4], rtol=1e-15)
        assert np.allclose(f[turns <= 1], base[turns <= 1] / 8, rtol=1e-15)
        mid = (turns > 1) & (turns < 4)
        assert mid.any() and np.all(f[mid] < base[mid]) and np.all(f[mid] > base[mid] / 8)
    for bad in (dict(rotary_dim=0), dict(rotary_dim=7), dict(rotary_dim=64, factor=0.5), dict(rotary_dim=64, scaling="x"),
                dict(rotary_dim=64, scaling="yarn"), dict(rotary_dim=64, scaling="yarn", original_ctx=10, low=4, high=2),
                dict(rotary_dim=2, scaling="ntk")):
        with pytest.raises(ValueError):
            kv.rope_frequencies(**bad)


def test_rope_init_refusals():
    assert kv.make_rope([]).rotary_dim == 0
    with pytest.raises(ValueError):
        kv.make_rope(np.ones(65))
    for f, kw, status in (([1.0] * 5, {}, UNS), ([math.nan] * 8, {}, INV), ([math.inf] * 8, {}, INV),
                          ([2.0 ** 21] * 8, {}, INV), ([1.0] * 8, dict(layout=2), INV),
                          ([1.0] * 8, dict(scale=math.nan), INV), ([1.0] * 8, dict(eps=-1.0), INV),
                          ([1.0] * 8, dict(eps=math.inf), INV)):
        with pytest.raises(kv.KVarNError) as e:
            kv.make_rope(f, **kw)
        assert e.value.status == status
    L, r = kv.lib(), kv.Rope()
    assert L.kvarn_rope_init(None, 16, 0, None, 1.0, 0.0) == INV
    assert L.kvarn_rope_init(ctypes.byref(r), 16, 0, None, 1.0, 0.0) == INV
    assert L.kvarn_rope_init(ctypes.byref(r), 144, 0, None, 1.0, 0.0) == INV


def _args(**change):
    """Arguments of kvarn_append_rope that pass every check but the ones changed (addresses are never read)."""
    cfg = kv.make_config(8, 2, 32, 2, synth.sign_bits(0))
    p = 0x10000
    a = dict(cfg=ctypes.byref(cfg), rope=ctypes.byref(kv.make_rope([1.0] * 8)), pool=p, n_pool=4, staging=p, table=p,
             max_blocks=4, pos=p, rope_pos=None, cu=None, n_tokens=2, batch=2, q=p, k=p, v=p, qs=1024, ks=256, vs=256,
             qw=None, kw=None, q_out=p, q_dtype=0, ws=p, stream=None)
    assert set(change) <= set(a)
    a.update(change)
    return list(a.values())


BAD = [dict(cfg=None), dict(rope=None), dict(pool=None), dict(pool=0x10008), dict(n_pool=-1), dict(n_pool=1 << 31),
       dict(table=None), dict(table=0x10002), dict(max_blocks=-1), dict(max_blocks=1 << 26), dict(pos=None),
       dict(pos=0x10001), dict(rope_pos=0x10002), dict(cu=0x10002), dict(n_tokens=3), dict(n_tokens=-1), dict(batch=-1),
       dict(k=None), dict(v=None), dict(q=None), dict(q_out=None), dict(k=0x10004), dict(q=0x10008), dict(qs=1023),
       dict(qs=1016), dict(ks=252), dict(ks=248), dict(vs=260), dict(qw=0x10004), dict(kw=0x10004), dict(q_out=0x10004),
       dict(q_dtype=2), dict(ws=None), dict(ws=0x10008), dict(cu=0x10000, n_tokens=1 << 40)]


@pytest.mark.parametrize("change", BAD, ids=[str(b) for b in BAD])
def test_append_rope_refusals(change):
    L, a = kv.lib(), _args(**change)
    assert L.kvarn_append_rope(*a) == INV
    del a[4]                                              # the same without staging
    assert L.kvarn_append_rope_bf16(*a) == INV


def test_append_rope_staging_refusals_and_empty_calls():
    L = kv.lib()
    for bad in (None, 0x10004):
        assert L.kvarn_append_rope(*_args(staging=bad)) == INV
    assert L.kvarn_append_rope(*_args(batch=0, n_tokens=0)) == 0
    assert L.kvarn_append_rope(*_args(cu=0x10000, n_tokens=0)) == 0
    r = kv.make_rope([1.0] * 8)
    r.rotary_dim = 24
    assert L.kvarn_append_rope(*_args(rope=ctypes.byref(r))) == UNS
