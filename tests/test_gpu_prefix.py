"""Shared-prefix decode attention against softmax in 64 bits over the same
cache bytes.

Tolerance, with p the softmax weights and all sums over a row's tokens. Packed
cache: query and key enter the score as three products of their bf16 halves,
each half pair within 2^-16 of its value (two roundings of 2^-8) and the
product of the low halves (2^-16) left out, so a score is within
d = 3 * 2^-16 * scale * sum_c |q_c k_c| (and fp32 sums of 128 terms, 2^-17); a
weight and a value are rounded to fp16 (2^-11 each) and so is the weight in
the normaliser: the output in the rotated space is within
(3 * 2^-11 + 2 d) sum p |v| of itself. A tile's values are scaled by the power
of two over its bound (largest (zero, top level) R times largest C), so small
ones keep an absolute half step of 2^-25 of at most twice the bound; weights
are held times 2^7, so one's absolute half step is 2^-32 of the largest, for
each of the n tokens. An unrotated channel is a sum of 128 of all that over
sqrt(128). bf16 cache: scores are fp32 sums of exact products
(d = 2^-17 scale sum |q k|), a weight is rounded to bf16 (2^-8, twice). The
2^-20 covers the fp32 merge. A bf16 output adds half a step, 2^-8 of itself.
"""
import math

import numpy as np
import pytest
import torch

import oracle
import synth
from kvtest_util import attn_close, bf16_bits

pytestmark = pytest.mark.gpu
D = 128


class Shared:
    """A pool with a prefix's blocks and each sequence's own, packed (bits) or bf16 (bits 0)."""

    def __init__(self, kv, seed, prefix, lens, n_q, n_kv, B, bits, flags=0, sm_scale=0.0, extra=0, wild=False, small=0):
        self.kv, self.bits, self.B, self.lens, self.prefix = kv, bits, B, list(lens), prefix
        self.sb = synth.sign_bits(seed)
        self.cfg = kv.make_config(n_q, n_kv, B, 2, self.sb, bits=bits or 2, flags=flags, sm_scale=sm_scale)
        self.scale = sm_scale or 1 / math.sqrt(D)
        g = synth.make_gen(seed, "cuda")
        batch, npb = len(lens), -(-prefix // B)
        nb = -(-max(lens) // B) if max(lens) else small
        self.n_pool = npb + batch * nb + 2 + extra
        ids = np.random.default_rng(seed).permutation(self.n_pool).astype(np.int32)
        if extra:
            ids = np.sort(ids)[::-1].copy()
        self.prefix_np, self.table_np = ids[:npb], ids[npb:npb + batch * nb].reshape(batch, nb)
        self.prefix_table, self.table = torch.from_numpy(self.prefix_np).cuda(), torch.from_numpy(self.table_np).cuda()
        kvs = (lambda n, L: synth.kv_values(g, n, n_kv, L, 1.5, 4, 20.0, "cuda")) if wild else \
            (lambda n, L: torch.randn(n, n_kv, L, D, generator=g, device="cuda"))
        P = torch.stack([kvs(1, npb * B)[0] for _ in range(2)], 1).to(torch.bfloat16)       # [n_kv][2][tokens][128]
        O = torch.stack([kvs(batch, nb * B) for _ in range(2)], 2).to(torch.bfloat16)       # [b][n_kv][2][tokens][128]
        self.staging = torch.zeros(batch, n_kv, 2, B, D, dtype=torch.bfloat16, device="cuda")
        blocks = torch.cat([P.unflatten(2, (npb, B)).permute(2, 0, 1, 3, 4),
                            O.unflatten(3, (nb, B)).permute(0, 3, 1, 2, 4, 5).flatten(0, 1)])
        where = torch.from_numpy(ids[:npb + batch * nb].astype(np.int64)).cuda()
        if bits == 0:
            self.pool = torch.full((self.n_pool, n_kv, 2, B, D), float("nan"), dtype=torch.bfloat16, device="cuda") \
                if not extra else torch.empty(self.n_pool, n_kv, 2, B, D, dtype=torch.bfloat16, device="cuda")
            self.pool[where] = blocks
            # what lies behind a sequence's end must not matter
            if prefix % B:
                self.pool[int(self.prefix_np[-1]), :, :, prefix % B:] = float("nan")
            for b, L in enumerate(lens):
                if L < nb * B:
                    self.pool[int(self.table_np[b, L // B]), :, :, L % B:] = float("nan")
        else:
            self.pool = torch.empty(self.n_pool, kv.block_bytes(self.cfg), dtype=torch.uint8, device="cuda")
            ws = kv.alloc_workspace(self.cfg, 0, 0)
            hb, bb = kv.head_block_bytes(self.cfg), kv.block_bytes(self.cfg)
            for h in range(n_kv):
                for kind in (0, 1):
                    kv.quantize_block(self.cfg, kind, blocks[:, h, kind].contiguous(), self.pool, ws,
                                      dst_offsets=where * bb + (2 * h + kind) * hb)
            for b, L in enumerate(lens):
                self.staging[b, :, :, :L % B] = O[b, :, :, L // B * B:L]
                self.staging[b, :, :, L % B:] = float("nan")
            assert kv.read_error(ws) == 0
        torch.cuda.synchronize()

    def i32(self, x):
        return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")

    def run(self, q, prefix_lens, seq_lens=None, out_dtype=torch.float32, ws=None, out=None, check=True):
        kv = self.kv
        out = torch.full(q.shape, 3.0, dtype=out_dtype, device="cuda") if out is None else out
        ws = kv.alloc_prefix_workspace(self.cfg, q.shape[0], len(self.prefix_np)) if ws is None else ws
        pl, sl = self.i32(prefix_lens), self.i32(self.lens if seq_lens is None else seq_lens)
        if self.bits:
            kv.prefix_attn(self.cfg, q, self.pool, self.staging, self.prefix_table, pl, self.table, sl, out, ws)
        else:
            kv.prefix_attn_bf16(self.cfg, q, self.pool, self.prefix_table, pl, self.table, sl, out, ws)
        if check:
            assert kv.read_error(ws) == 0
        return out

    def _bound(self, ids, h):
        """Largest (|zero|, |top level|) R times largest C of the V head-blocks."""
        hb = self.kv.head_block_bytes(self.cfg)
        raw = self.pool[torch.from_numpy(ids.astype(np.int64)).cuda()][:, (2 * h + 1) * hb:(2 * h + 2) * hb].cpu().numpy()
        top = lambda f: (np.maximum(np.abs(f["z16"]), np.abs(f["z16"] + (2 ** self.bits - 1) * f["s16"]))  # noqa: E731
                         * f["R16"][:, None]).max() * np.abs(f["C16"]).max()
        return max([top(oracle.unpack(self.B, 1, np.ascontiguousarray(r), bits=self.bits)) for r in raw] + [0.0])

    def _head(self, ids, h):
        if not self.bits:
            t = self.pool[torch.from_numpy(ids.astype(np.int64)).cuda()][:, h].double().cpu().numpy()
            return t[:, 0].reshape(-1, D), t[:, 1].reshape(-1, D)
        hb = self.kv.head_block_bytes(self.cfg)
        raw = self.pool[torch.from_numpy(ids.astype(np.int64)).cuda()][:, 2 * h * hb:(2 * h + 2) * hb].cpu().numpy()
        return [oracle.decode_blocks(np.ascontiguousarray(raw[:, k * hb:(k + 1) * hb]), self.B, k, self.sb, True,
                                     flags=int(self.cfg.flags) & 7, bits=self.bits).reshape(-1, D) for k in (0, 1)]

    def reference(self, q, prefix_lens, seqs=None):
        """(out, tolerance before the output's rounding) of the chosen sequences, float64 [len(seqs)][n_q][128]."""
        n_q, n_kv, B = self.cfg.n_q_heads, self.cfg.n_kv_heads, self.B
        G = n_q // n_kv
        seqs = range(q.shape[0]) if seqs is None else seqs
        rot = bool(self.bits) and not int(self.cfg.flags) & 1
        turn = (lambda x: oracle.rotate(x, self.sb)) if rot else (lambda x: x)
        H = oracle.hadamard() / math.sqrt(D)
        qn = q.double().cpu().numpy()
        stg = self.staging.double().cpu().numpy()
        want, tol = np.zeros((len(seqs), n_q, D)), np.zeros((len(seqs), n_q, D))
        for h in range(n_kv):
            kp, vp = self._head(self.prefix_np, h)
            bound = self._bound(self.prefix_np, h) if self.bits else 0.0
            for i, b in enumerate(seqs):
                L, P = self.lens[b], prefix_lens[b]
                whole = L // B * B if self.bits else L
                ks, vs = [kp[:P]], [vp[:P]]
                if whole:
                    ko, vo = self._head(self.table_np[b], h)
                    ks.append(ko[:whole])
                    vs.append(vo[:whole])
                if L > whole:
                    ks.append(turn(stg[b, h, 0, :L - whole]))
                    vs.append(turn(stg[b, h, 1, :L - whole]))
                k, v = np.concatenate(ks), np.concatenate(vs)
                if not len(k):
                    continue
                qr = turn(qn[b, h * G:(h + 1) * G])
                s = qr @ k.T * self.scale
                p = np.exp(s - s.max(-1, keepdims=True))
                p /= p.sum(-1, keepdims=True)
                o, A = p @ v, p @ np.abs(v)
                size = (np.abs(qr) @ np.abs(k).T * self.scale).max(-1, keepdims=True)
                d = ((3 * 2.0 ** -16 if self.bits else 0) + 2.0 ** -17) * size
                d = np.minimum(np.expm1(np.minimum(2 * d, 1.0)), 2.0)
                t = ((3 * 2.0 ** -11 if self.bits else 2 * 2.0 ** -8) + d + 2.0 ** -20) * A
                t = t + (2.0 ** -24 + P * 2.0 ** -32) * bound
                if rot:
                    o = o @ H * oracle.sigma(self.sb)
                    t = np.repeat(t.sum(-1, keepdims=True) / math.sqrt(D), D, -1)
                want[i, h * G:(h + 1) * G], tol[i, h * G:(h + 1) * G] = o, t
        return want, tol


def _close(got, want, tol):
    got64 = got.double().cpu().numpy()
    if got.dtype == torch.bfloat16:
        tol = tol * (1 + 2.0 ** -8) + np.abs(want) * 2.0 ** -8
    err = np.abs(got64 - want)
    assert np.all(np.isfinite(got64)) and np.all(err <= tol + 1e-30), float((err / (tol + 1e-30)).max())


CASES = [  # prefix, prefix_lens (None: all), own lengths, n_q, n_kv, B, q dtype, out dtype
    (1, None, [0], 1, 1, 32, torch.bfloat16, torch.float32),
    (100, [0, 1, 31, 100, 17, 64], [0, 0, 32, 3, 69, 1], 8, 2, 32, torch.bfloat16, torch.bfloat16),
    (300, None, [5 + i % 70 for i in range(40)], 8, 2, 64, torch.float32, torch.float32),
    (129, [129 - i for i in range(65)], [1] * 65, 3, 1, 64, torch.bfloat16, torch.float32),
    (2049, [2049, 2048, 0, 777], [0, 0, 0, 0], 6, 3, 64, torch.bfloat16, torch.bfloat16),
    (640, [640] * 70 + [3], [33] * 71, 8, 2, 32, torch.bfloat16, torch.float32),
    (4100, [4100, 4099], [200, 1], 40, 10, 32, torch.float32, torch.bfloat16),
    (0, [0, 0], [40, 7], 4, 1, 32, torch.bfloat16, torch.float32),
    (9000, None, [64, 0, 31], 2, 2, 64, torch.bfloat16, torch.float32),
]


@pytest.mark.parametrize("bits", [0, 2, 3, 4])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_against_64_bits(kvlib, case, bits):
    prefix, pl, lens, n_q, n_kv, B, qdt, odt = CASES[case]
    s = Shared(kvlib, 20 + case, prefix, lens, n_q, n_kv, B, bits)
    pl = [prefix] * len(lens) if pl is None else pl
    q = (2 * synth.queries(synth.make_gen(case), len(lens), n_q)).to(qdt).cuda()
    got = s.run(q, pl, out_dtype=odt)
    seqs = sorted(set(list(range(min(6, len(lens)))) + [len(lens) // 2, len(lens) - 1]))
    want, tol = s.reference(q, pl, seqs)
    _close(got[seqs], want, tol)
    assert torch.equal(got, s.run(q, pl, out_dtype=odt))           # the same bits every time
    for b in range(len(lens)):
        if pl[b] == 0 and lens[b] == 0:
            assert torch.all(got[b] == 0)


@pytest.mark.parametrize("bits,B", [(0, 32), (2, 32), (2, 64), (4, 64)])
def test_outlier_keys_and_sharp_softmax(kvlib, bits, B):
    """Lognormal token scales and outlier channels (the workloads' value model): scores in the hundreds."""
    lens = [70, 3, 0, 129]
    s = Shared(kvlib, 7 + B, 515, lens, 8, 2, B, bits, wild=True)
    q = synth.queries(synth.make_gen(3), 4, 8).to(torch.bfloat16).cuda()
    pl = [515, 400, 515, 1]
    want, tol = s.reference(q, pl)
    _close(s.run(q, pl), want, tol)


@pytest.mark.parametrize("bits", [0, 2, 3, 4])
@pytest.mark.parametrize("batch,n_q,n_kv,B,P", [(256, 40, 10, 64, 2300), (8, 128, 64, 32, 2600), (70, 96, 48, 64, 3333)])
def test_many_tiles_for_each_range(kvlib, bits, batch, n_q, n_kv, B, P):
    """More row tiles and heads than the GPU has SMs: each CTA walks 10 to 50 tiles, whose value exponents differ."""
    lens = [i % 3 for i in range(batch)]
    s = Shared(kvlib, 31, P, lens, n_q, n_kv, B, bits, wild=True)
    q = synth.queries(synth.make_gen(4), batch, n_q).to(torch.bfloat16).cuda()
    pl = [P - 7 * (i % 5) for i in range(batch)]
    got = s.run(q, pl)
    seqs = [0, batch // 2, batch - 1]
    want, tol = s.reference(q, pl, seqs)
    _close(got[seqs], want, tol)
    for _ in range(5):
        assert torch.equal(got, s.run(q, pl))


@pytest.mark.parametrize("bits", [0, 2])
def test_scale_and_ablation_flags(kvlib, bits):
    for flags, scale in ((kvlib.FLAG_NO_ROTATION, 0.0), (0, 0.5), (kvlib.FLAG_NO_TOKEN_PASS, 0.02)):
        s = Shared(kvlib, 9, 200, [3, 65], 4, 2, 32, bits, flags=flags if bits else 0, sm_scale=scale)
        q = synth.queries(synth.make_gen(5), 2, 4).cuda()
        want, tol = s.reference(q, [200, 150])
        _close(s.run(q, [200, 150]), want, tol)


@pytest.mark.parametrize("bits", [0, 2])
def test_equals_decode_over_joined_tables(kvlib, bits):
    """With whole blocks, one table of the prefix's and the own blocks through the plain decode attention."""
    kv, B, P = kvlib, 64, 512
    lens = [130, 64, 5]
    s = Shared(kv, 11, P, lens, 16, 4, B, bits)
    q = synth.queries(synth.make_gen(6), 3, 16).to(torch.bfloat16).cuda()
    got = s.run(q, [P] * 3)
    table = torch.cat([s.prefix_table[None].expand(3, -1), s.table], 1).contiguous()
    ws = kv.alloc_workspace(s.cfg, 3, table.shape[1])
    out, sl = torch.empty(3, 16, D, device="cuda"), s.i32([P + L for L in lens])
    if bits:
        kv.decode_attn(s.cfg, q, s.pool, s.staging, table, sl, out, ws)
    else:
        kv.decode_attn_bf16(s.cfg, q, s.pool, table, sl, out, ws)
    attn_close(got.double().cpu().numpy(), out.double().cpu().numpy())


@pytest.mark.parametrize("bits", [0, 3])
def test_faults_are_flagged(kvlib, bits):
    kv = kvlib
    s = Shared(kv, 13, 200, [70, 3, 40], 8, 2, 32, bits)
    q = synth.queries(synth.make_gen(7), 3, 8).cuda()
    ws = kv.alloc_prefix_workspace(s.cfg, 3, len(s.prefix_np))
    good = s.run(q, [200] * 3, ws=ws)
    assert kv.read_error(ws) == 0
    for pl, sl in (([200, -1, 200], None), ([200, 225, 200], None), ([2 ** 31 - 1, 200, 200], None),
                   ([200] * 3, [70, -1, 40]), ([200] * 3, [97, 3, 40])):
        kv.clear_error(ws)
        got = s.run(q, pl, sl, ws=ws, check=False)
        assert kv.read_error(ws) == kv.DEVERR_POSITION
        for b in range(3):
            if pl[b] == 200 and (sl is None or sl[b] == s.lens[b]):
                assert torch.equal(got[b], good[b])
            else:
                assert torch.isnan(got[b]).all()
    for bad in (-1, s.n_pool, 2 ** 31 - 1, -2 ** 31):
        kept = int(s.prefix_table[3])
        s.prefix_table[3] = bad
        kv.clear_error(ws)
        s.run(q, [200] * 3, ws=ws, check=False)
        assert kv.read_error(ws) == kv.DEVERR_BLOCK_ID
        s.prefix_table[3] = kept
    kv.clear_error(ws)
    assert torch.equal(s.run(q, [200] * 3, ws=ws), good)


@pytest.mark.parametrize("bits,batch", [(0, 3), (0, 80), (2, 3), (2, 80), (4, 80)])
def test_wait_timeout_path(kvlib, bits, batch):
    """With the test switch the prefix kernels' product warp leaves at once: the other warps follow, the flag is raised,
    and the workspace serves the next call."""
    kv = kvlib
    s = Shared(kv, 33, 1500, [2] * batch, 8, 2, 64, bits)
    q = synth.queries(synth.make_gen(2), batch, 8).to(torch.bfloat16).cuda()
    ws = kv.alloc_prefix_workspace(s.cfg, batch, len(s.prefix_np))
    good = s.run(q, [1500] * batch, ws=ws)
    s.cfg.flags |= kv.FLAG_TEST_WAIT_TIMEOUT
    for _ in range(3):
        s.run(q, [1500] * batch, ws=ws, check=False)
        assert kv.read_error(ws) == kv.DEVERR_WAIT_TIMEOUT
        kv.clear_error(ws)
    s.cfg.flags &= ~kv.FLAG_TEST_WAIT_TIMEOUT
    assert torch.equal(s.run(q, [1500] * batch, ws=ws), good)


@pytest.mark.parametrize("bits", [0, 2])
def test_pool_beyond_4_gib(kvlib, bits):
    n_kv, B = 2, 64
    per = n_kv * 2 * (B * D * 2 if bits == 0 else 3456)
    s = Shared(kvlib, 15, 190, [66, 1], 4, n_kv, B, bits, extra=(1 << 32) // per + 5)
    q = synth.queries(synth.make_gen(8), 2, 4).cuda()
    want, tol = s.reference(q, [190, 100])
    _close(s.run(q, [190, 100]), want, tol)


@pytest.mark.parametrize("bits", [0, 2])
def test_two_graphs_with_their_own_workspaces(kvlib, bits):
    """Captured calls replayed at once on two streams, lengths changed between replays."""
    kv = kvlib
    s = Shared(kv, 17, 700, [100, 31, 64], 8, 2, 32, bits)
    q = [synth.queries(synth.make_gen(20 + i), 3, 8).cuda() for i in range(2)]
    pl, sl = s.i32([700, 650, 3]), s.i32(s.lens)
    ws = [kv.alloc_prefix_workspace(s.cfg, 3, len(s.prefix_np)) for _ in range(2)]
    outs = [torch.zeros(3, 8, D, device="cuda") for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]

    def call(i):
        if bits:
            kv.prefix_attn(s.cfg, q[i], s.pool, s.staging, s.prefix_table, pl, s.table, sl, outs[i], ws[i])
        else:
            kv.prefix_attn_bf16(s.cfg, q[i], s.pool, s.prefix_table, pl, s.table, sl, outs[i], ws[i])

    for i in range(2):
        call(i)
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for i in range(2):
        with torch.cuda.graph(graphs[i], stream=streams[i]):
            call(i)
    for lens in ([700, 650, 3], [1, 0, 699]):
        pl.copy_(s.i32(lens))
        torch.cuda.synchronize()
        for _ in range(3):
            for i in range(2):
                with torch.cuda.stream(streams[i]):
                    graphs[i].replay()
        torch.cuda.synchronize()
        for i in range(2):
            assert kv.read_error(ws[i]) == 0
            assert torch.equal(outs[i], s.run(q[i], lens))


OWN = [  # own lengths, batch repeats, n_q, n_kv, B, q dtype
    ([1024, 1023, 0, 517, 16, 15, 1, 64], 1, 8, 2, 64, torch.bfloat16),
    ([1024, 33, 992, 0], 1, 3, 1, 32, torch.float32),
    ([700, 5, 0, 128, 300], 1, 4, 2, 64, torch.float32),
    ([90, 129, 17, 64, 255, 1], 4, 28, 7, 64, torch.bfloat16),     # more units than the GPU has SMs
    ([40, 3, 100, 0, 63], 13, 12, 12, 32, torch.float32),          # several waves of them
    ([2048, 31, 0, 1999, 1], 1, 12, 4, 64, torch.bfloat16),
    ([2047, 1100], 1, 2, 2, 32, torch.float32),
    ([1500, 2048] + [3] * 78, 1, 4, 4, 64, torch.bfloat16),        # long ones among many
]


@pytest.mark.parametrize("bits", [0, 2, 3, 4])
@pytest.mark.parametrize("case", range(len(OWN)))
def test_own_tokens_in_narrow_and_wide_tables(kvlib, case, bits):
    """Own tokens up to 2048; the same with table columns that no length reaches, for which other kernels serve."""
    lens, times, n_q, n_kv, B, qdt = OWN[case]
    lens, P = lens * times, 150
    s = Shared(kvlib, 50 + case, P, lens, n_q, n_kv, B, bits)
    q = (2 * synth.queries(synth.make_gen(30 + case), len(lens), n_q)).to(qdt).cuda()
    pl = [(P, 0, 149, 1)[b % 4] for b in range(len(lens))]
    seqs = list(range(len(lens) // times)) + [len(lens) - 1]
    want, tol = s.reference(q, pl, seqs)
    table = s.table
    for columns in sorted({max(c, table.shape[1]) for c in (0, 1024 // B + 1, 2048 // B, 2048 // B + 1, 4096 // B)}):
        s.table = torch.full((len(lens), columns), -1, dtype=torch.int32, device="cuda")
        s.table[:, :table.shape[1]] = table
        got = s.run(q, pl)
        _close(got[seqs], want, tol)
        assert torch.equal(got, s.run(q, pl))


@pytest.mark.parametrize("bits", [0, 2])
def test_bad_own_blocks_are_flagged(kvlib, bits):
    """A bad entry of a sequence's own table touches no other sequence and reads nothing."""
    kv = kvlib
    s = Shared(kv, 61, 100, [200, 70, 300], 8, 2, 32, bits)
    q = synth.queries(synth.make_gen(7), 3, 8).cuda()
    narrow = s.table
    for columns in (narrow.shape[1], 80):
        s.table = torch.full((3, columns), -1, dtype=torch.int32, device="cuda")
        s.table[:, :narrow.shape[1]] = narrow
        ws = kv.alloc_prefix_workspace(s.cfg, 3, len(s.prefix_np))
        good = s.run(q, [100, 3, 0], ws=ws)
        for bad in (-1, s.n_pool, 2 ** 31 - 1, -2 ** 31):
            kept = int(s.table[0, 2])
            s.table[0, 2] = bad
            got = s.run(q, [100, 3, 0], ws=ws, check=False)
            assert kv.read_error(ws) == kv.DEVERR_BLOCK_ID
            assert torch.equal(got[1:], good[1:])
            s.table[0, 2] = kept
            kv.clear_error(ws)
        assert torch.equal(s.run(q, [100, 3, 0], ws=ws), good)


@pytest.mark.parametrize("bits,columns", [(0, 4), (0, 80), (2, 4), (2, 80)])
def test_inputs_that_the_kernel_before_wrote(kvlib, bits, columns):
    """Lengths, table entries, queries and own rows written on the stream just before each call, with nothing waited for:
    the same bits as with the GPU idle between the steps."""
    s = Shared(kvlib, 71, 640, [120] * 6, 8, 2, 32, bits)
    gen, steps = synth.make_gen(12), 60
    qs = torch.stack([synth.queries(gen, 6, 8) for _ in range(steps)]).to(torch.bfloat16).cuda()
    narrow, pool, staging = s.table, s.pool.clone(), s.staging.clone()
    rows = torch.randn(steps, *s.staging.shape[:3], D, generator=torch.Generator("cuda").manual_seed(3), device="cuda").to(torch.bfloat16)
    ws = kvlib.alloc_prefix_workspace(s.cfg, 6, len(s.prefix_np))
    results = []
    for wait in (True, False):
        s.pool.copy_(pool)
        s.staging.copy_(staging)
        table = torch.full((6, columns), -1, dtype=torch.int32, device="cuda")
        q, pl, sl = torch.zeros_like(qs[0]), s.i32([0] * 6), s.i32([0] * 6)
        outs = torch.zeros(steps, 6, 8, D, device="cuda")
        for i in range(steps):
            L = 2 * i + 1
            q.copy_(qs[i])
            table[:, (L - 1) // 32] = narrow[:, (L - 1) // 32]
            sl.add_(L - (2 * i - 1 if i else 0))
            pl.add_(10)
            if bits:
                s.staging[:, :, :, (L - 1) % 32] = rows[i]
                if L % 32:
                    s.staging[:, :, :, :L % 32].nan_to_num_(0.25)
            else:
                page = s.pool[narrow[:, (L - 1) // 32].long()]
                page[:, :, :, (L - 1) % 32] = rows[i]
                s.pool[narrow[:, (L - 1) // 32].long()] = page
            if wait:
                torch.cuda.synchronize()
            if bits:
                kvlib.prefix_attn(s.cfg, q, s.pool, s.staging, s.prefix_table, pl, table, sl, outs[i], ws)
            else:
                kvlib.prefix_attn_bf16(s.cfg, q, s.pool, s.prefix_table, pl, table, sl, outs[i], ws)
        torch.cuda.synchronize()
        assert kvlib.read_error(ws) == 0
        results.append(outs)
    assert torch.isfinite(results[0]).all()
    assert torch.equal(results[0], results[1])


def test_no_own_blocks_and_small_tables(kvlib):
    for bits in (0, 2):
        s = Shared(kvlib, 19, 64, [0, 0], 4, 2, 32, bits)           # a block table without columns
        q = synth.queries(synth.make_gen(9), 2, 4).cuda()
        want, tol = s.reference(q, [64, 0])
        got = s.run(q, [64, 0])
        _close(got, want, tol)
        assert torch.all(got[1] == 0)


@pytest.mark.parametrize("n_q,n_kv,B", [(32, 8, 64), (40, 10, 32), (1, 1, 64), (128, 64, 32)])
@pytest.mark.parametrize("batch", [1, 5, 64, 700])
def test_a_workspace_serves_shorter_prefixes(kvlib, n_q, n_kv, B, batch):
    cfg = kvlib.make_config(n_q, n_kv, B, 2, synth.sign_bits(1))
    sizes = [kvlib.prefix_workspace_bytes(cfg, batch, b) for b in list(range(0, 400)) + [512, 1000, 4096, 20000]]
    assert all(0 < x <= y for x, y in zip(sizes, sizes[1:]))


def test_workspace_and_binding_refusals(kvlib):
    kv = kvlib
    s = Shared(kv, 19, 64, [40, 3], 4, 2, 32, 2)
    q = synth.queries(synth.make_gen(9), 2, 4).cuda()
    n = kv.prefix_workspace_bytes(s.cfg, 2, 2)
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    s.run(q, [64, 1], ws=ws)
    with pytest.raises(kv.KVarNError) as e:
        s.run(q, [64, 1], ws=ws[:n - 16])
    assert e.value.status == -4
    out, pl, sl = torch.zeros(2, 4, D, device="cuda"), s.i32([64, 1]), s.i32([40, 3])
    good = dict(cfg=s.cfg, q=q, pool=s.pool, staging=s.staging, prefix_table=s.prefix_table, prefix_lens=pl,
                block_table=s.table, seq_lens=sl, out=out, workspace=ws)
    kv.prefix_attn(**good)
    for bad in (dict(q=q[:1].contiguous()), dict(q=q.half()), dict(out=out[:, :2].contiguous()), dict(out=out.half()),
                dict(prefix_lens=pl[:1]), dict(seq_lens=sl.long()), dict(block_table=s.table[:1]),
                dict(staging=s.staging[:1]), dict(pool=s.pool[:, 16:].contiguous()), dict(prefix_table=s.prefix_table.cpu())):
        with pytest.raises(ValueError):
            kv.prefix_attn(**{**good, **bad})


@pytest.mark.parametrize("packed", [False, True])
def test_a_serving_step_from_prompt_to_shared_decode(kvlib, packed):
    """The operators as they are used together: a shared prompt appended once, each sequence's own tokens appended
    behind it at their positions in the whole text, and decode attention over both, against the whole text's attention
    in 64 bits over the rotated keys. bf16 pages: each key carries half a bf16 step (2^-8), so a score is off by at most
    2^-8 scale sum |q k| on top of the kernel's own. Packed: 4-bit codes are compared over the cache's own values."""
    kv = kvlib
    n_q, n_kv, B, P, lens = 8, 2, 32, 150, [45, 7, 70]
    f = kv.rope_frequencies(128, 10000.0)[0]
    rope = kv.make_rope(f)
    cfg = kv.make_config(n_q, n_kv, B, 2, synth.sign_bits(2), bits=4)
    g = torch.Generator().manual_seed(1)
    rows = lambda n: torch.randn(n, (n_q + 2 * n_kv) * D, generator=g).to(torch.bfloat16).cuda()  # noqa: E731
    cut = lambda x: [y.unflatten(1, (-1, D)) for y in x.split([n_q * D, n_kv * D, n_kv * D], 1)]  # noqa: E731
    npb, nb = 160 // B, 4
    n_pool = npb + 3 * nb
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    ptab = torch.arange(npb, dtype=torch.int32, device="cuda")
    table = torch.arange(npb, n_pool, dtype=torch.int32, device="cuda").view(3, nb)
    ws = kv.alloc_prefix_workspace(cfg, 3, npb)
    shared = 150 if not packed else 128          # packed: only complete blocks can be shared, the rest is each one's own
    prompt = rows(P)
    if packed:
        pool, stage = kv.alloc_pool(cfg, n_pool), kv.alloc_staging(cfg, 3)
        pstage = kv.alloc_staging(cfg, 1)
        put = lambda tab, st, *a, **k: kv.append_rope(cfg, rope, pool, st, tab, *a, **k)  # noqa: E731
    else:
        pool, stage, pstage = torch.zeros(n_pool, n_kv, 2, B, D, dtype=torch.bfloat16, device="cuda"), None, None
        put = lambda tab, st, *a, **k: kv.append_rope_bf16(cfg, rope, pool, tab, *a, **k)  # noqa: E731
    _, k, v = cut(prompt[:shared])
    put(ptab[None], pstage, i32([0]), None, k, v, None, ws, cu_tokens=i32([0, shared]))
    # each sequence: the prompt's rest and its own tokens in one ragged run, then one more token as a decode step
    own = [torch.cat([prompt[shared:], rows(n - 1)]) for n in lens]
    cu = np.concatenate([[0], np.cumsum([len(o) for o in own])])
    q, k, v = cut(torch.cat(own))
    put(table, stage, i32([0, 0, 0]), None, k, v, None, ws, cu_tokens=i32(cu), rope_pos=i32([shared] * 3))
    last = rows(3)
    q, k, v = cut(last)
    n_own = [len(o) for o in own]
    q_out = torch.empty(3, n_q, D, device="cuda")
    put(table, stage, i32(n_own), q, k, v, q_out, ws, rope_pos=i32([shared + n for n in n_own]))
    out = torch.empty(3, n_q, D, device="cuda")
    a = (ptab, i32([shared] * 3), table, i32([n + 1 for n in n_own]), out, ws)
    if packed:
        kv.prefix_attn(cfg, q_out, pool, stage, *a)
    else:
        kv.prefix_attn_bf16(cfg, q_out, pool, *a)
    assert kv.read_error(ws) == 0
    if packed:   # the joined tables through the plain decode attention read the same bytes
        joined = torch.cat([ptab[:shared // B][None].expand(3, -1), table], 1).contiguous()
        ref = torch.empty_like(out)
        kv.decode_attn(cfg, q_out, pool, stage, joined, i32([shared + n + 1 for n in n_own]), ref,
                       kv.alloc_workspace(cfg, 3, joined.shape[1]))
        attn_close(out.double().cpu().numpy(), ref.double().cpu().numpy())
        return

    def turned(x, pos):
        x = x.double().cpu().numpy()
        ang = np.asarray(pos, np.float64)[:, None] * f
        c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]
        return np.concatenate([x[..., :64] * c - x[..., 64:] * s, x[..., 64:] * c + x[..., :64] * s], -1)

    for b in range(3):
        text = torch.cat([prompt[:shared], own[b], last[b:b + 1]])
        qa, ka, va = cut(text)
        n = len(text)
        kk, vv = turned(ka, np.arange(n)), va.double().cpu().numpy()
        qq = turned(qa[-1:], [n - 1])[0]
        for hq in range(n_q):
            kh, vh = kk[:, hq // 4], vv[:, hq // 4]
            sc = kh @ qq[hq] / math.sqrt(D)
            p = np.exp(sc - sc.max())
            p /= p.sum()
            d = (2.0 ** -8 + 2.0 ** -15) * (np.abs(kh) @ np.abs(qq[hq])).max() / math.sqrt(D)
            tol = (2 * 2.0 ** -8 + math.expm1(2 * d) + 2.0 ** -20) * (p @ np.abs(vh))
            assert np.all(np.abs(out[b, hq].double().cpu().numpy() - p @ vh) <= tol)
