"""Tree attention where the parts of a sum differ by many powers of two, over blocks
whose factors are written here and whose values are therefore known.

Bounds, relative to a weight of 1 of the row's largest, from kvarn.h:
  weights   two fp16 halves: 2^-22 of themselves and 2^-36; two bf16 halves 2^-16 (the
            few-rows kernel 2^-22 and, by its block's own scale, 2^-38)
  scores    (2^-17 + 2^-20 + 2^-16) of |q| |k| scale, as in cache_util; a weight and the
            sum it is divided by each move by that
  sums      the tensor core adds 16 tokens a step, three products of halves, and may cut
            a sum at 2^-23 of itself: 3 N / 16 of those. Weights below 2^-25 of what
            the sum already holds may be lost.
  ex2.approx, sums of weights, merge and division: 2^-15 with the weights' halves
"""
import math

import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu
D = 128
SCALE = 1 / math.sqrt(D)


def _pool(kv, cfg, bits, kinds):
    """Blocks of one kv head: kinds = (K, V), each (codes or None, step, zero, R), step, zero and R [tokens]; C is 1."""
    B = cfg.block_size
    hb, x = kv.head_block_bytes(cfg), 16 * bits * B
    n = len(kinds[0][1]) // B
    p = np.zeros((n, 2, hb), np.uint8)

    def put(kind, at, v):
        v = np.ascontiguousarray(v, np.float16)
        p[:, kind, at:at + 2 * v.shape[1]] = v.view(np.uint8).reshape(n, -1)

    for kind, (codes, step, zero, r) in enumerate(kinds):
        if codes is not None:
            p[:, kind, :x] = codes.integers(0, 256, (n, x), dtype=np.uint8)
        put(kind, x, np.tile(step.reshape(n, 1, B), (1, 4, 1)).reshape(n, -1))
        put(kind, x + 8 * B, np.tile(zero.reshape(n, 1, B), (1, 4, 1)).reshape(n, -1))
        put(kind, x + 16 * B, r.reshape(n, B))
        put(kind, x + 18 * B, np.ones((n, D)))
    return p


def _tree(kv, cfg, bits, pool, q, N, batch):
    """The cached tokens' attention of every row (no draft is shown to any), the same table for all sequences."""
    T, B = q.shape[1], cfg.block_size
    table = torch.arange(N // B, dtype=torch.int32, device="cuda").repeat(batch, 1).contiguous()
    lens = torch.full((batch,), N, dtype=torch.int32, device="cuda")
    k = torch.zeros(batch, T, 1, D, dtype=torch.bfloat16, device="cuda")
    mask = torch.zeros(batch, T, (T + 31) // 32, dtype=torch.int32, device="cuda")
    out = torch.zeros(q.shape, device="cuda")
    ws = kv.alloc_tree_workspace(cfg, batch, T, N // B)
    if bits:
        kv.tree_attn(cfg, q, pool, kv.alloc_staging(cfg, batch), table, lens, k, k, mask, out, ws)
    else:
        kv.tree_attn_bf16(cfg, q, pool, table, lens, k, k, mask, out, ws)
    assert kv.read_error(ws) == 0
    return out.double().cpu().numpy()


@pytest.mark.parametrize("value", [0.0, 1.0])
@pytest.mark.parametrize("below", [22.6, 24.5, 26.4, 27.6, 28.05])
@pytest.mark.parametrize("bits,T", [(2, 7), (4, 7), (2, 33), (3, 3), (0, 7)])
def test_many_small_weights_beside_a_large_one(kvlib, bits, T, below, value):
    """Token 5 has most of the attention; the others, 2^-below of it each, make the output where its value is zero. A
    sequence for each SM, so that one CTA has all of a sequence's tokens (two, of bf16 pages)."""
    kv = kvlib
    N, B, G = 16384, 64, 4
    batch = torch.cuda.get_device_properties(0).multi_processor_count
    cfg = kv.make_config(G, 1, B, 2, [0] * 4, bits=bits or 2, flags=kv.FLAG_NO_ROTATION)
    keys, values = np.zeros(N), 0.75 + 0.125 * (np.arange(N) % 5)
    keys[5], values[5] = 1.0, value
    if bits:
        none, one = np.zeros(N), np.ones(N)
        pool = torch.from_numpy(_pool(kv, cfg, bits, ((None, none, one, keys), (None, none, one, values))).reshape(N // B, -1)).cuda()
    else:
        both = torch.from_numpy(np.stack([keys, values])).to(torch.bfloat16).view(2, N // B, 1, B, 1)
        pool = both.permute(1, 2, 0, 3, 4).expand(N // B, 1, 2, B, D).contiguous().cuda()
    each = np.float32(below * math.log(2) / (D * SCALE))
    q = torch.full((batch, T, G, D), float(each), device="cuda")
    out = _tree(kv, cfg, bits, pool, q, N, batch)

    score = float(each) * D * SCALE
    w = math.exp(-score)
    small = values.sum() - value
    want = (value + w * small) / (1 + w * (N - 1))
    d = (2.0 ** -17 + 2.0 ** -20 + 2.0 ** -16) * score
    allowed = (math.exp(2 * d) - 1 + 2.0 ** -15 + 3 * N / 16 * 2.0 ** -23) * want + 2.0 ** -36 * small
    if value:
        allowed += w * small * (w < 2.0 ** -24)   # (lost beside a sum of 1)
    assert np.abs(out - want).max() <= allowed, (np.abs(out - want).max(), allowed, want)


@pytest.mark.parametrize("bits", [2, 3, 4])
@pytest.mark.parametrize("down", [0, 8, 12, 20])
def test_small_values_in_a_tile_with_a_large_one(kvlib, bits, down):
    """Of 64 tokens one is 2^down times as large as the others, and none of the attention goes to it. Keys and values are within
    2^-18 of their token's largest level, or 2^-29 of the tile's."""
    kv = kvlib
    N, B, G, T = 256, 32, 4, 7
    cfg = kv.make_config(G, 1, B, 2, [0] * 4, bits=bits, flags=kv.FLAG_NO_ROTATION)
    top = 2 ** bits - 1
    large = np.arange(N) % 64 == 37
    keys = np.where(large, -1.0, 0.0)
    reach = np.where(large, 1.0, 2.0 ** -down)     # (R: levels run from -reach to reach)
    step, zero = np.full(N, 2 / top, np.float16), np.full(N, -1.0)
    none, one = np.zeros(N), np.ones(N)
    raw = _pool(kv, cfg, bits, ((None, none, one, keys), (np.random.default_rng(3), step, zero, reach)))
    values = oracle.decode_blocks(np.ascontiguousarray(raw[:, 1]), B, 1, [0] * 4, False, flags=1, bits=bits).reshape(-1, D)
    q = torch.full((3, T, G, D), 100 / (D * SCALE), device="cuda")
    out = _tree(kv, cfg, bits, torch.from_numpy(raw.reshape(N // B, -1)).cuda(), q, N, 3)
    want = values[~large].mean(0)                  # (weights of e^-100 are nothing)
    size = np.abs(values[~large]).mean(0)
    allowed = (2.0 ** -15 + 3 * N / 16 * 2.0 ** -23) * size + 2.0 ** -18 * 2.0 ** -down * 1.01 + 2.0 ** -29
    assert (np.abs(out - want).max((0, 1, 2)) <= allowed).all(), (np.abs(out - want).max((0, 1, 2)) / allowed).max()
