"""A paged cache for the tests of the long-generation operators: sequences of any
lengths in scattered blocks, packed or bf16, and what a token stands for in 64 bits.

Error of a softmax output, for the tolerances of those tests. Let d_t bound the
error of token t's score (natural units), p the weights, D = sum p_t d_t. A weight
p_t = exp(s_t) / sum exp(s) then grows by at most r_t = exp(d_t + D), for the normaliser
shrinks to no less than sum p exp(-d) >= exp(-D) of itself; where it is held as
two 16-bit halves or comes from ex2.approx it is off by another e_p of itself. An
output, a sum of p_t v_t, has a 2-norm off by at most sum_t p_t (r_t - 1 + e_p) |v_t|.
2-norms do not change under the rotation of the packed cache.
  d_t: a score is a sum of 128 products in fp32 (2^-24 a step: 2^-17 in all) of
  factors that may be split into two halves (two fp16 halves 2^-22, two bf16 halves,
  of an fp32 query alone, 2^-16): at most (2^-17 + 2^-20 [+ 2^-16]) scale |q| e_t.
  e_t = |k_t|; of packed blocks the 2-norm of (|z| + top s) R C, because codes times
  steps and zeros are summed apart. The same extent takes the place of |v_t|.
  e_p: 2^-16 for two bf16 halves, 2^-20 for ex2.approx, the merge and the division:
  together 2^-15 at most.
"""
import math

import numpy as np
import torch

import oracle
import synth

D = 128


class Cache:
    """lens tokens of each sequence; bits 0: bf16 pages. What lies behind a
    sequence's end, in pages and in staging, is NaN. `extra` free blocks lie
    before the used ones, `spare` free ones are left for other tables."""

    def __init__(self, kv, seed, lens, n_q, n_kv, B, bits, flags=0, sm_scale=0.0, wild=False, blocks=None, extra=0, spare=0):
        self.kv, self.bits, self.B, self.lens, self.n_kv = kv, bits, B, [int(L) for L in lens], n_kv
        self.sb = synth.sign_bits(seed)
        self.cfg = kv.make_config(n_q, n_kv, B, 2, self.sb, bits=bits or 2, flags=flags, sm_scale=sm_scale)
        self.scale = sm_scale or 1 / math.sqrt(D)
        g = synth.make_gen(seed, "cuda")
        batch = len(lens)
        nb = -(-max(lens) // B) if blocks is None else blocks
        used = batch * nb
        self.n_pool = used + spare + extra + 1
        ids = extra + np.random.default_rng(seed).permutation(used + spare + 1).astype(np.int32)
        self.table_np, self.spare_np = ids[:used].reshape(batch, nb), ids[used:used + spare]
        self.table = torch.from_numpy(self.table_np).cuda()
        self.seq_lens = i32(self.lens)
        shape = (batch, n_kv, 2, nb * B, D)
        if wild:
            raw = torch.stack([synth.kv_values(g, batch, n_kv, nb * B, 1.5, 4, 20.0, "cuda") for _ in range(2)], 2)
        else:
            raw = torch.randn(*shape, generator=g, device="cuda")
        raw = raw.to(torch.bfloat16)                                              # [b][n_kv][2][tokens][128]
        blk = raw.unflatten(3, (nb, B)).permute(0, 3, 1, 2, 4, 5).flatten(0, 1)      # [b nb][n_kv][2][B][128]
        where = torch.from_numpy(self.table_np.reshape(-1).astype(np.int64)).cuda()
        self.staging = torch.full((batch, n_kv, 2, B, D), float("nan"), dtype=torch.bfloat16, device="cuda")
        if bits == 0:
            self.pool = torch.empty(self.n_pool, n_kv, 2, B, D, dtype=torch.bfloat16, device="cuda")
            if not extra:
                self.pool.fill_(float("nan"))
            self.pool[where] = blk
            for b, L in enumerate(self.lens):
                if L < nb * B:
                    self.pool[int(self.table_np[b, L // B]), :, :, L % B:] = float("nan")
        else:
            hb, bb = kv.head_block_bytes(self.cfg), kv.block_bytes(self.cfg)
            self.pool = torch.empty(self.n_pool, bb, dtype=torch.uint8, device="cuda")
            ws = kv.alloc_workspace(self.cfg, 0, 0)
            if used:
                for h in range(n_kv):
                    for kind in (0, 1):
                        kv.quantize_block(self.cfg, kind, blk[:, h, kind].contiguous(), self.pool, ws,
                                          dst_offsets=where * bb + (2 * h + kind) * hb)
            for b, L in enumerate(self.lens):
                self.staging[b, :, :, :L % B] = raw[b, :, :, L // B * B:L]
            assert kv.read_error(ws) == 0
        torch.cuda.synchronize()

    def tokens(self, b, h, L=None, table=None, staging_of=None):
        """fp64 ([K, V] each [L][128], [extent of K, of V] each [L]) of the first L tokens of sequence b."""
        L = self.lens[b] if L is None else L
        ids = torch.from_numpy((self.table_np if table is None else table)[b].astype(np.int64)).cuda()
        B, bits = self.B, self.bits
        if bits == 0:
            t = self.pool[ids[:-(-L // B)], h].double().cpu().numpy()
            vals = [t[:, k].reshape(-1, D)[:L] for k in (0, 1)]
            return vals, [np.linalg.norm(x, axis=1) for x in vals]
        n, hb = L // B, self.kv.head_block_bytes(self.cfg)
        raw = self.pool[ids[:n], 2 * h * hb:2 * (h + 1) * hb].cpu().numpy()
        tail = self.staging[b if staging_of is None else staging_of, h, :, :L % B].double().cpu().numpy()
        vals, extents = [], []
        for kind in (0, 1):
            mine = np.ascontiguousarray(raw[:, kind * hb:(kind + 1) * hb])
            val = oracle.decode_blocks(mine, B, kind, self.sb, False, flags=int(self.cfg.flags) & 7, bits=bits).reshape(-1, D)
            f = np.ascontiguousarray(mine[:, 16 * bits * B:]).view(np.float16).astype(np.float64)
            step, zero = f[:, :4 * B].reshape(n, 4, B), f[:, 4 * B:8 * B].reshape(n, 4, B)
            reach = (np.abs(zero) + (2 ** bits - 1) * step).repeat(32, 1).transpose(0, 2, 1)   # [n][B][128]
            reach = reach * f[:, 8 * B:9 * B, None] * f[:, None, 9 * B:]
            vals.append(np.concatenate([val, tail[kind]]))
            extents.append(np.concatenate([np.linalg.norm(reach, axis=2).reshape(-1), np.linalg.norm(tail[kind], axis=1)]))
        return vals, extents


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def attend(q, K, V, ek, ev, scale, q32, shown=None):
    """(out [rows][128], bound of its rows' 2-norm error, weights p, bounds of their errors) in 64 bits, of query rows
    q over tokens K, V with extents ek, ev; shown [rows][tokens]."""
    s = scale * (q @ K.T)
    if shown is not None:
        s = np.where(shown, s, -np.inf)
    top = s.max(1, keepdims=True, initial=-np.inf)
    w = np.exp(s - np.where(np.isinf(top), 0.0, top))
    total = w.sum(1, keepdims=True)
    p = w / np.where(total > 0, total, 1.0)
    d = (2.0 ** -17 + 2.0 ** -20 + (2.0 ** -16 if q32 else 0.0)) * scale * np.linalg.norm(q, axis=1)[:, None] * ek
    Dn = (p * d).sum(1, keepdims=True)
    off = p * (np.exp(np.minimum(d + Dn, 40)) - 1 + 2.0 ** -15)
    return p @ V, off @ ev, p, off


def close_rows(got, want, tol, bf16):
    """Rows of fp64 `got` within the 2-norm bounds; a bf16 output adds half a step of itself."""
    err = np.linalg.norm(got - want, axis=-1)
    allowed = tol + (2.0 ** -8 * np.linalg.norm(want, axis=-1) if bf16 else 2.0 ** -22 * np.linalg.norm(want, axis=-1))
    assert np.isfinite(got).all()
    worst = (err / np.maximum(allowed, 1e-300)).max(initial=0.0) if np.any(allowed > 0) else 0.0
    assert (err <= allowed).all(), f"worst error {worst:.3g} of its bound"
    return worst
