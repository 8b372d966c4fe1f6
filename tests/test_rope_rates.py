"""The rotary rates as fractions of a turn: exact to the unit whatever the size
and sign of the rate, and the rotation at far positions that rests on it."""
import random
from fractions import Fraction

import numpy as np
import pytest
import torch

import bit_kv_cache_08_gb300 as kv
import synth

# pi to 60 digits
PI = Fraction(3141592653589793238462643383279502884197169399375105820974944, 10 ** 60)
D = 128


def _turns(rate):
    """rate / (2 pi) mod 1 (60 digits of pi leave 2^-180)."""
    return Fraction(rate) / (2 * PI) % 1


def test_rates_of_every_size_are_exact_to_the_unit():
    """Half a unit of 2^-64 from the rounding, and 2^-75: the constant's 2^-108 of up to 2^18 turns, and the rounding of
    the remainder (below 2^-35) and of the last sum (below 2^33 units)."""
    kv.build()
    r = random.Random(7)
    rates = [0.0, 1.0, -1.0, 2.0 ** 20, -2.0 ** 20, 5e-324, -5e-324, 1e-300, -1e-17, 1e-17, 2.0 ** -40, 1048575.999]
    rates += [r.choice((-1, 1)) * 2.0 ** r.uniform(-45, 20) for _ in range(4084)]
    for i in range(0, len(rates), 64):
        part = rates[i:i + 64]
        got = kv.make_rope(part).turns
        for x, t in zip(part, got):
            d = (Fraction(t, 1 << 64) - _turns(x)) % 1
            assert min(d, 1 - d) <= Fraction(1, 1 << 65) + Fraction(1, 1 << 75), x


@pytest.mark.gpu
@pytest.mark.parametrize("rate", [1.0, 37.5, 1000.0, -70000.25, 2.0 ** 20])
def test_rotation_at_far_positions(kvlib, rate):
    """Positions to either end of 32 bits: the angle is within 2^-33 turns of the formula's (a unit's half times the
    position), pi 2^-25 and sincospif's 2 ulp on top, so within 1e-6 (|a| + |b|) as at position 0."""
    cfg = kvlib.make_config(1, 1, 64, 2, synth.sign_bits(0))
    far = [2 ** 31 - 1, -2 ** 31, 2 ** 30 + 12345, -7, 0, 99999999]
    n, pairs = len(far), 64
    f = rate * (1 - np.arange(pairs) / 100)
    x = torch.randn(n, 1, D, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16).cuda()
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    pool = torch.zeros(n, 1, 2, 64, D, dtype=torch.bfloat16, device="cuda")
    out = torch.empty(n, 1, D, device="cuda")
    ws = kvlib.alloc_workspace(cfg, 0, 0)
    kvlib.append_rope_bf16(cfg, kvlib.make_rope(f), pool, i32([[i] for i in range(n)]), i32([0] * n), x, x, x, out, ws,
                           rope_pos=i32(far))
    assert kvlib.read_error(ws) == 0
    ang = np.array([[float(_turns(float(w)) * p % 1) for w in f] for p in far]) * 2 * np.pi
    a, b = x[:, 0, :pairs].double().cpu().numpy(), x[:, 0, pairs:].double().cpu().numpy()
    want = np.concatenate([a * np.cos(ang) - b * np.sin(ang), b * np.cos(ang) + a * np.sin(ang)], 1)
    err = np.abs(out[:, 0].double().cpu().numpy() - want)
    tol = 1e-6 * np.tile(np.abs(a) + np.abs(b), 2) + 2.0 ** -24 * np.abs(want)
    print("largest error over its tolerance:", float((err / tol).max()))
    assert np.all(err <= tol)
