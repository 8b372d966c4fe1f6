"""How many bits the shared-prefix attention keeps: fp32 outputs against the
same softmax in 64 bits over the same cache bytes, row by row in the 2-norm
(which the rotation back leaves as it is), so that what one 16-bit rounding of
a weight, a value, a key or a query costs does not hide behind a sum over 128
channels.

Tolerance of a row, t_c = e A_c for channel c of the space the products run in,
A = sum p |v|, and the 2-norm of t plus 2^-20 of the output's (8 fp32 roundings
of the rotation back and the store), with e the sum of
  what is kept of a weight and a value   2^-16 for a weight in bf16 halves (a
    bf16 value is exact), 3 * 2^-22 in fp16 halves (a weight, a value, and the
    product of the low halves, which is left out)
  the scores   2 d: a score is off by d, its weight by that, and the normaliser
    by it again; d = (2^-17 for the fp32 sum of 128 products, 2^-22 for the
    exponent's product and sum, and 2^-16 for an fp32 query in bf16 halves)
    times scale sum |q_c k_c|
  2^-18   at most 16 accumulations of 16 tokens' products for a range of at
    most 128 tokens and half, each within 2^-23, the exponential's 2^-22, the
    normaliser's sum and the merge
"""
import math

import numpy as np
import pytest
import torch

import oracle
import synth
from test_gpu_prefix import Shared

pytestmark = pytest.mark.gpu
D = 128


def _exact(s, q, pl):
    """(output, A, largest scale sum |q k|) of every row, float64, in the space of the products; own tokens: none."""
    n_q, n_kv = s.cfg.n_q_heads, s.cfg.n_kv_heads
    G = n_q // n_kv
    rot = bool(s.bits) and not int(s.cfg.flags) & 1
    qn = q.double().cpu().numpy()
    o, A, size = np.zeros(qn.shape), np.zeros(qn.shape), np.zeros(qn.shape[:2] + (1,))
    for h in range(n_kv):
        kp, vp = s._head(s.prefix_np, h)
        for b, P in enumerate(pl):
            k, v, at = kp[:P], vp[:P], (b, slice(h * G, (h + 1) * G))
            qr = oracle.rotate(qn[at], s.sb) if rot else qn[at]
            x = qr @ k.T * s.scale
            p = np.exp(x - x.max(-1, keepdims=True))
            p /= p.sum(-1, keepdims=True)
            o[at], A[at] = p @ v, p @ np.abs(v)
            size[at] = (np.abs(qr) @ np.abs(k).T * s.scale).max(-1, keepdims=True)
    return o, A, size


def _check(s, q, pl, kept, score):
    o, A, size = _exact(s, q, pl)
    got = s.run(q, pl).double().cpu().numpy()
    if s.bits and not int(s.cfg.flags) & 1:
        got = oracle.rotate(got, s.sb).reshape(got.shape)
    tol = (kept + 2.0 ** -18 + np.expm1(2 * score * size)) * A
    norm = lambda x: np.linalg.norm(x, axis=-1)  # noqa: E731
    ratio = norm(got - o) / (norm(tol) + 2.0 ** -20 * norm(o))
    print("largest error over its tolerance:", float(ratio.max()))
    assert np.all(np.isfinite(got)) and ratio.max() <= 1.0


CASES = [  # prefix tokens, batch, n_q, n_kv, B, q dtype
    (2, 3, 4, 4, 32, torch.bfloat16),
    (5, 40, 8, 2, 64, torch.bfloat16),
    (5, 40, 8, 2, 64, torch.float32),
    (40, 150, 4, 4, 32, torch.bfloat16),
    (40, 7, 3, 1, 32, torch.float32),
    (128, 70, 8, 4, 64, torch.bfloat16),
]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_weights_over_bf16_pages(kvlib, case):
    """Flat scores, so that every weight counts and none is a power of two."""
    P, batch, n_q, n_kv, B, qdt = CASES[case]
    s = Shared(kvlib, 80 + case, P, [0] * batch, n_q, n_kv, B, 0, small=1)
    q = (0.1 * synth.queries(synth.make_gen(40 + case), batch, n_q)).to(qdt).cuda()
    score = 2.0 ** -17 + 2.0 ** -22 + (2.0 ** -16 if qdt == torch.float32 else 0)
    _check(s, q, [P] * batch, 2.0 ** -16, score)


PACKED = [  # prefix tokens, batch, n_q, n_kv, B, q dtype
    (2, 3, 4, 4, 32, torch.bfloat16),
    (5, 40, 8, 2, 64, torch.bfloat16),
    (33, 150, 4, 4, 32, torch.float32),
    (64, 70, 8, 4, 64, torch.bfloat16),
    (90, 5, 3, 1, 32, torch.bfloat16),
]


@pytest.mark.parametrize("bits", [2, 3, 4])
@pytest.mark.parametrize("case", range(len(PACKED)))
def test_weights_and_values_over_the_packed_cache(kvlib, case, bits):
    """Flat scores; the queries so small that what the score's halves leave out (3 * 2^-16 of sum |q k|) is nothing."""
    P, batch, n_q, n_kv, B, qdt = PACKED[case]
    s = Shared(kvlib, 90 + case, P, [0] * batch, n_q, n_kv, B, bits, small=1)
    q = (0.01 * synth.queries(synth.make_gen(50 + case), batch, n_q)).to(qdt).cuda()
    # (a weight and a value as fp16 pairs: 2^-22 each and the product of the low halves)
    _check(s, q, [P] * batch, 3 * 2.0 ** -22, 3 * 2.0 ** -16 + 2.0 ** -17)


@pytest.mark.parametrize("bits,B,batch", [(2, 32, 6), (3, 64, 40), (4, 32, 40), (4, 64, 6)])
@pytest.mark.parametrize("qdt", [torch.float32, torch.bfloat16])
def test_scores_over_the_packed_cache(kvlib, bits, B, batch, qdt):
    """Scores of one product each (queries of one channel, no rotation) and up to 60: no sum hides what the halves of a
    key and of a query leave out. As fp16 pairs that is 2^-22 each and the product of the low halves; 2^-22 for the
    exponent's product and sum."""
    P = 96
    s = Shared(kvlib, 100 + bits, P, [0] * batch, 8, 2, B, bits, flags=kvlib.FLAG_NO_ROTATION, small=1)
    g = torch.Generator().manual_seed(bits)
    q = torch.zeros(batch, 8, D)
    q.scatter_(2, torch.randint(0, D, (batch, 8, 1), generator=g), 150 * (1 + torch.rand(batch, 8, 1, generator=g)))
    _check(s, q.to(qdt).cuda(), [P] * batch, 3 * 2.0 ** -22, 2.0 ** -20)
