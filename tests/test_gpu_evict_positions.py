"""Rotary positions in a cache that eviction has cut down: a place is then no position, and appends take rope_pos."""
import numpy as np
import pytest
import torch

from cache_util import Cache, attend, close_rows, i32

pytestmark = pytest.mark.gpu
D = 128


@pytest.mark.parametrize("bits,B", [(0, 32), (0, 64), (2, 32), (4, 64)])
def test_appends_after_evictions(kvlib, bits, B):
    """Two rounds of an eviction, a run of tokens and single ones, beside a cache that is never cut: with rope_pos the
    new keys and queries are those of the uncut cache bit for bit, and what is attended to is what was kept."""
    kv = kvlib
    n_q, n_kv, budget, recent = 8, 2, 2 * B, B
    G = n_q // n_kv
    lens = [5 * B + 9, 3 * B, B + 5]
    batch, blocks = len(lens), 9
    rope = kv.make_rope(kv.rope_frequencies(D)[0])
    cut, whole = (Cache(kv, 90, lens, n_q, n_kv, B, bits, blocks=blocks, spare=2 * batch * blocks) for _ in range(2))
    pages = cut.spare_np.reshape(2, batch, blocks)
    g = torch.Generator(device="cuda").manual_seed(8)
    ws = kv.alloc_weights_workspace(cut.cfg, batch, blocks)
    at = i32(lens)                                   # positions of the next tokens
    where = [[np.arange(L) for _ in range(n_kv)] for L in lens]   # the position of each place

    def append(c, q, k, v, counts, rope_pos=None):
        cu = i32(np.concatenate([[0], np.cumsum(counts)]))
        q_out = torch.zeros(q.shape, dtype=torch.float32, device="cuda")
        if bits:
            kv.append_rope(c.cfg, rope, c.pool, c.staging, c.table, c.seq_lens, q, k, v, q_out, ws, cu_tokens=cu, rope_pos=rope_pos)
        else:
            kv.append_rope_bf16(c.cfg, rope, c.pool, c.table, c.seq_lens, q, k, v, q_out, ws, cu_tokens=cu, rope_pos=rope_pos)
        c.seq_lens = c.seq_lens + i32(counts)
        c.lens = c.seq_lens.tolist()
        return q_out

    for turn in range(2):
        weights = torch.rand(batch, n_kv, blocks * B, generator=g, device="cuda")
        new_table = torch.from_numpy(pages[turn]).cuda()
        new_lens, new_weights = torch.zeros_like(cut.seq_lens), torch.zeros_like(weights)
        kept = torch.zeros(batch, n_kv, budget // B if bits else budget, dtype=torch.int32, device="cuda")
        (kv.evict if bits else kv.evict_bf16)(cut.cfg, cut.pool, cut.table, cut.seq_lens, weights, new_table, new_lens, new_weights,
                                              kept, ws, budget=budget, recent=recent)
        unit = B if bits else 1
        for b in range(batch):
            for h in range(n_kv):
                x = kept[b, h].cpu().numpy()
                x = (x[x >= 0][:, None] * unit + np.arange(unit)).ravel()
                where[b][h] = np.concatenate([where[b][h][x], where[b][h][cut.lens[b] - cut.lens[b] % unit:]])
        cut.table, cut.table_np, cut.seq_lens, cut.lens = new_table, pages[turn], new_lens, new_lens.tolist()
        for counts in ([7, 0, B + 3], [1, 1, 1], [1, 1, 1]):
            n = sum(counts)
            q, k, v = (torch.randn(n, m, D, generator=g, device="cuda").to(torch.bfloat16) for m in (n_q, n_kv, n_kv))
            got = append(cut, q, k, v, counts, rope_pos=at)
            want = append(whole, q, k, v, counts)
            assert torch.equal(got, want)
            at = at + i32(counts)
            for b in range(batch):
                for h in range(n_kv):
                    where[b][h] = np.concatenate([where[b][h], np.arange(whole.lens[b] - counts[b], whole.lens[b])])
            assert whole.lens == at.tolist()
        # every place holds the key and value of its position in the uncut cache
        for b in range(batch):
            for h in range(n_kv):
                (K, V), _ = cut.tokens(b, h)
                (K0, V0), _ = whole.tokens(b, h)
                assert (K == K0[where[b][h]]).all() and (V == V0[where[b][h]]).all()
        out = torch.zeros(batch, n_q, D, device="cuda")
        w = torch.zeros_like(weights)
        if bits:
            kv.decode_attn_weights(cut.cfg, got, cut.pool, cut.staging, cut.table, cut.seq_lens, out, w, ws, decay=0.0)
        else:
            kv.decode_attn_weights_bf16(cut.cfg, got, cut.pool, cut.table, cut.seq_lens, out, w, ws, decay=0.0)
        for b in range(batch):
            for h in range(n_kv):
                (K, V), (ek, ev) = cut.tokens(b, h)
                qb, ob = (x[b, h * G:(h + 1) * G].double().cpu().numpy() for x in (got, out))
                expect, tol, _, _ = attend(qb, K, V, ek, ev, cut.scale, True)
                close_rows(ob, expect, tol, False)
        assert kv.read_error(ws) == 0
