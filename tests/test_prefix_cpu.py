"""Argument checks and sizes of the shared-prefix attention (nothing is launched)."""
import ctypes

import pytest

import bit_kv_cache_08_gb300 as kv
import synth

INV = -1


@pytest.fixture(scope="module", autouse=True)
def built():
    kv.build()


def _args(**change):
    """Arguments of kvarn_prefix_attn that pass every check but the ones changed (addresses are never read)."""
    cfg = kv.make_config(8, 2, 32, 2, synth.sign_bits(0))
    p = 0x10000
    a = dict(cfg=ctypes.byref(cfg), q=p, q_dtype=0, pool=p, n_pool=4, staging=p, ptable=p, pblocks=2, plens=p, table=p,
             max_blocks=4, lens=p, batch=2, out=p, out_dtype=1, ws=p, ws_bytes=1 << 30, stream=None)
    assert set(change) <= set(a)
    a.update(change)
    return list(a.values())


BAD = [dict(cfg=None), dict(q=None), dict(q=0x10004), dict(q_dtype=2), dict(pool=None), dict(pool=0x10008),
       dict(n_pool=0), dict(n_pool=1 << 31), dict(ptable=None), dict(ptable=0x10002), dict(pblocks=-1),
       dict(pblocks=1 << 27), dict(pblocks=(1 << 25) + 1), dict(plens=None), dict(plens=0x10001), dict(table=None), dict(table=0x10002),
       dict(max_blocks=-1), dict(max_blocks=1 << 27), dict(lens=None), dict(lens=0x10002), dict(batch=-1),
       dict(batch=1 << 30), dict(out=None), dict(out=0x10004), dict(out_dtype=2), dict(ws=None), dict(ws=0x10008)]


@pytest.mark.parametrize("change", BAD, ids=[str(b) for b in BAD])
def test_refusals(change):
    L, a = kv.lib(), _args(**change)
    assert L.kvarn_prefix_attn(*a) == INV
    del a[5]                                              # the same without staging
    assert L.kvarn_prefix_attn_bf16(*a) == INV


def test_tensors_of_another_device_are_refused(monkeypatch):
    """The binding compares every tensor's device with the current one (two stand-in devices)."""
    class OnDevice:
        device = "cuda:1"

        def __init__(self, i):
            self.i = i

        def get_device(self):
            return self.i

    monkeypatch.setattr(kv._abi, "_raw_device", lambda: 0)
    kv._abi._need_device(OnDevice(0), None, OnDevice(0))
    with pytest.raises(ValueError):
        kv._abi._need_device(OnDevice(0), OnDevice(1))


def test_staging_and_empty_batch():
    L = kv.lib()
    for bad in (None, 0x10008):
        assert L.kvarn_prefix_attn(*_args(staging=bad)) == INV
    assert L.kvarn_prefix_attn(*_args(batch=0)) == 0
    cfg = kv.make_config(8, 2, 32, 2, synth.sign_bits(0))
    assert kv.prefix_workspace_bytes(cfg, 0, 10) == 256
    assert kv.prefix_workspace_bytes(cfg, 1, (1 << 25) + 1) == 0 and kv.prefix_workspace_bytes(cfg, 1 << 29, 1) == 0
    assert kv.prefix_workspace_bytes(cfg, -1, 10) == 0 and kv.prefix_workspace_bytes(cfg, 1, -1) == 0
