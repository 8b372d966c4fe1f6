"""The serving step around the paged caches, as cases to be measured: appending
a step's keys and values with the head norms and the position rotation on the
way, and decode attention for a batch that shares a prompt.

Two kinds of case (``op``), each for both caches (``cache``: "bf16" pages, or
"packed" head-blocks of 2-, 3- or 4-bit codes with a bf16 staging buffer):

append   q, k, v come as columns of one projection's rows. q and k get an RMS
         norm per head (where ``norm``) and the rotary rotation of the token's
         position; k and v go to the token's place in the cache, q to q_out.
         A packed case writes the staging rows of tokens inside a block.
prefix   softmax(q k / sqrt(128)) v over the first prefix_lens[b] tokens of a
         prefix that all sequences share, followed by seq_lens[b] own tokens.

``own`` selects the plain torch form (False) or the package's kernels (True).
"""
import math

import numpy as np
import torch

own = False

D = 128
_MASK = {2: 3, 3: 7, 4: 15}


# ------------------------------------------------------------------ cases

def _append(name, cache, batch, tokens, n_q, n_kv, block, rotary, layout, norm, theta, far):
    return dict(name=name, op="append", cache=cache, batch=batch, tokens=tokens, n_q=n_q, n_kv=n_kv, block=block,
                rotary=rotary, layout=layout, norm=norm, theta=theta, far=far)


def _prefix(name, cache, batch, prefix, ctx, n_q, n_kv, block, bits):
    return dict(name=name, op="prefix", cache=cache, batch=batch, prefix=prefix, ctx=ctx, n_q=n_q, n_kv=n_kv,
                block=block, bits=bits)


def listed():
    return [
        # one user's next token: the latency of a call
        _append("append-bf16-1tok", "bf16", 1, 1, 32, 8, 32, 128, "half", False, 500000.0, 0),
        # a decode step of the benchmark's batch, with head norms
        _append("append-bf16-64tok", "bf16", 64, 1, 32, 8, 64, 128, "half", True, 1000000.0, 0),
        # a few ragged prompts; interleaved pairs over three quarters of the head, far along a long context
        _append("append-bf16-prompts-odd", "bf16", 7, 201, 40, 10, 32, 96, "interleaved", False, 10000.0, 100003),
        # a prefill batch of ragged prompts
        _append("append-bf16-prompts-32k", "bf16", 24, 1365, 32, 8, 64, 128, "half", True, 1000000.0, 0),
        # decode steps over the packed cache: the benchmark's batch, and a small one with part of the head rotated
        _append("append-packed-64tok", "packed", 64, 1, 32, 8, 64, 128, "half", True, 1000000.0, 0),
        _append("append-packed-8tok", "packed", 8, 1, 40, 10, 32, 96, "half", False, 10000.0, 16384),
        # a handful of requests over a short system prompt
        _prefix("prefix-bf16-4x1k", "bf16", 4, 1000, 64, 32, 8, 32, 2),
        # an ordinary batch over a long system prompt
        _prefix("prefix-bf16-64x8k", "bf16", 64, 8192, 256, 32, 8, 64, 2),
        # many samples of one long document
        _prefix("prefix-bf16-128x32k", "bf16", 128, 32768, 512, 32, 8, 64, 2),
        # the same three uses over the packed cache
        _prefix("prefix-2bit-5x1k", "packed", 5, 1111, 70, 32, 8, 32, 2),
        _prefix("prefix-2bit-64x8k", "packed", 64, 8192, 256, 32, 8, 64, 2),
        _prefix("prefix-4bit-128x32k", "packed", 128, 32768, 512, 32, 8, 64, 4),
    ]


def _log(rng, lo, hi):
    """A whole number from lo to hi, spread over its logarithm."""
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    cache = rng.choice(["bf16", "packed"])
    n_kv = rng.choice([1, 2, 3, 4, 8, 10])
    group = rng.choice([1, 2, 3, 4])
    block = rng.choice([32, 64])
    if rng.random() < 0.5:
        batch = _log(rng, 1, 192)
        tokens = 1 if cache == "packed" or rng.random() < 0.4 else _log(rng, 2, max(2, min(2000, 30000 // batch)))
        c = _append("", cache, batch, tokens, n_kv * group, n_kv, block, rng.choice([16, 32, 64, 96, 128]),
                    rng.choice(["half", "interleaved"]), rng.random() < 0.5, rng.choice([10000.0, 500000.0, 1000000.0]),
                    rng.choice([0, 0, _log(rng, 1, 1000000)]))
    else:
        batch = _log(rng, 1, 128)
        ctx = _log(rng, 1, 600)
        c = _prefix("", cache, batch, _log(rng, 1, 32768), ctx, n_kv * group, n_kv, block, rng.choice([2, 3, 4]))
    del c["name"]
    return c


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    r = np.random.RandomState(int(seed) % (1 << 31))
    return dict(case=case, **(_prepare_append if case["op"] == "append" else _prepare_prefix)(case, g, r))


def _ints(values):
    return torch.tensor(np.asarray(values), dtype=torch.int32, device="cuda")


def _prepare_append(c, g, r):
    batch, n_q, n_kv, B = c["batch"], c["n_q"], c["n_kv"], c["block"]
    most = c["tokens"]
    # prompts: half to one and a half of `tokens` each, batch * tokens in all; a decode step: one
    more = r.randint(0, most // 2 + 1, batch // 2)
    counts = most + np.concatenate([more, -more, np.zeros(batch % 2, np.int64)])
    counts = r.permutation(counts)
    cached = r.randint(0, 4 * B, batch)
    if c["cache"] == "packed":   # a token that does not complete its block: staging alone is written
        cached -= cached % B == B - 1
    cu = np.concatenate([[0], np.cumsum(counts)])
    T = int(cu[-1])
    nb = -(-(4 * B + most + most // 2) // B)
    n_pool = batch * nb + 3
    rows = torch.randn(T, (n_q + 2 * n_kv) * D, generator=g, device="cuda", dtype=torch.float32)
    rows *= torch.exp(0.5 * torch.randn(T, 1, generator=g, device="cuda"))
    rows = rows.to(torch.bfloat16)
    s = dict(
        q=rows[:, :n_q * D].view(T, n_q, D), k=rows[:, n_q * D:(n_q + n_kv) * D].view(T, n_kv, D),
        v=rows[:, (n_q + n_kv) * D:].view(T, n_kv, D), rows=rows,
        q_weight=None, k_weight=None, pos=_ints(cached), rope_pos=_ints(cached + c["far"]),
        cu_tokens=None if most == 1 else _ints(cu), n_pool=n_pool,
        block_table=_ints(r.permutation(n_pool)[:batch * nb].reshape(batch, nb)),
        inv_freq=c["theta"] ** (-np.arange(0, c["rotary"], 2, dtype=np.float64) / c["rotary"]),
        q_out=torch.empty(T, n_q, D, dtype=torch.bfloat16, device="cuda"))
    s["freq"] = torch.from_numpy(s["inv_freq"]).cuda()
    if c["norm"]:
        for name in ("q_weight", "k_weight"):
            s[name] = (1 + 0.3 * torch.randn(D, generator=g, device="cuda")).to(torch.bfloat16)
    if c["cache"] == "bf16":
        s["pool"] = torch.randn(n_pool, n_kv, 2, B, D, generator=g, device="cuda", dtype=torch.bfloat16)
    else:
        s["staging"] = torch.randn(batch, n_kv, 2, B, D, generator=g, device="cuda", dtype=torch.bfloat16)
    return s


def _block_bytes(B, bits):
    return (16 * bits + 18) * B + 256


def _packed_pool(n, n_kv, B, bits, g):
    """n physical blocks: random codes, and steps, zeros and factors like those of quantised keys and values."""
    hb, x = _block_bytes(B, bits), 16 * bits * B
    levels = (1 << bits) - 1
    pool = torch.empty(n, n_kv, 2, hb, dtype=torch.uint8, device="cuda")
    pool[..., :x] = torch.randint(0, 256, (n, n_kv, 2, x), generator=g, device="cuda", dtype=torch.uint8)

    def put(at, values):
        v = values.to(torch.float16).contiguous()
        pool[..., at:at + v.shape[-1] * 2] = v.view(torch.uint8).view(n, n_kv, 2, -1)

    reach = 1.5 + torch.rand(n, n_kv, 2, 4 * B, generator=g, device="cuda")   # a group's values lie within -reach .. reach
    put(x, 2 * reach / levels)
    put(x + 8 * B, -reach)
    put(x + 16 * B, torch.exp(0.4 * torch.randn(n, n_kv, 2, B, generator=g, device="cuda")))
    put(x + 18 * B, torch.exp(0.4 * torch.randn(n, n_kv, 2, D, generator=g, device="cuda")))
    return pool.view(n, -1)


def _prepare_prefix(c, g, r):
    batch, n_q, n_kv, B, P, ctx = c["batch"], c["n_q"], c["n_kv"], c["block"], c["prefix"], c["ctx"]
    lens = r.randint(max(1, ctx // 2), ctx + 1, batch)
    shared = np.full(batch, P)
    if batch > 2:   # one sequence left the prefix early, one does not use it
        shared[r.randint(1, batch)] = r.randint(0, P + 1)
        shared[0] = 0
    npb, nb = -(-P // B), -(-ctx // B)
    n_pool = npb + batch * nb + 2
    pages = r.permutation(n_pool)
    s = dict(q=(2 * torch.randn(batch, n_q, D, generator=g, device="cuda")).to(torch.bfloat16),   # scores of a few units
             prefix_table=_ints(pages[:npb]), prefix_lens=_ints(shared),
             block_table=_ints(pages[npb:npb + batch * nb].reshape(batch, nb)), seq_lens=_ints(lens), n_pool=n_pool,
             out=torch.empty(batch, n_q, D, dtype=torch.bfloat16, device="cuda"))
    if c["cache"] == "bf16":
        s["pool"] = torch.randn(n_pool, n_kv, 2, B, D, generator=g, device="cuda", dtype=torch.bfloat16)
        s["pool"] *= torch.exp(0.4 * torch.randn(1, n_kv, 2, 1, D, generator=g, device="cuda")).to(torch.bfloat16)
    else:
        s["pool"] = _packed_pool(n_pool, n_kv, B, c["bits"], g)
        s["staging"] = torch.randn(batch, n_kv, 2, B, D, generator=g, device="cuda").to(torch.bfloat16)
        s["sign_bits"] = [int(w) for w in r.randint(0, 1 << 32, 4, dtype=np.uint64)]
        signs = [1.0 - 2.0 * ((s["sign_bits"][i // 32] >> (i % 32)) & 1) for i in range(D)]
        s["signs"] = torch.tensor(signs, device="cuda")
        s["places"] = _places(B, c["bits"])
        s["hadamard"] = _hadamard(torch.float32) / math.sqrt(D)
    return s


def _places(B, bits):
    """Word and bit of each (token, channel) code within a head-block, for K and V; 3-bit codes also those of the high bit."""
    t, ch = np.arange(B)[:, None], np.arange(D)[None, :]
    g = ch // 32
    found = []
    for kind in (0, 1):
        if kind == 0:
            a, i, b, e = t % 32 // 4, t % 4, ch % 32 // 8, ch % 8
            w, j, h = 2 * i + g // 2, 4 * (g % 2) + e // 2, e % 2
            if bits == 4:
                w, j = 4 * i + g, e // 2
        else:
            b, d, a, f = t % 32 // 8, t % 8, ch % 32 // 4, ch % 4
            w, j, h = 2 * g + f // 2, 4 * (d // 4) + 2 * (d % 4 // 2) + f % 2, d % 2
            if bits == 4:
                w, j = 4 * g + f, d // 2
        rec = 32 * (t // 32) + 4 * a + b
        wide = 4 if bits == 4 else 2
        one = [rec * 4 * bits + w, wide * j + 16 * h]
        one += [rec * 12 + 8 + w // 2, 8 * (w % 2) + j + 16 * h] if bits == 3 else one
        found.append(np.stack([np.broadcast_to(x, (B, D)) for x in one]))
    return torch.from_numpy(np.stack(found)).cuda()   # [kind][4][B][128]


# ------------------------------------------------------------------ one pass

def run(state):
    if own:
        return _own(state)
    return _plain_append(state) if state["case"]["op"] == "append" else _plain_prefix(state)


def _own(s):
    import bit_kv_cache_08_gb300 as kv
    c = s["case"]
    if "cfg" not in s:   # what a program sets up once for its model and batch
        s["cfg"] = kv.make_config(c["n_q"], c["n_kv"], c["block"], 2, s.get("sign_bits", [0, 0, 0, 0]),
                                  bits=c.get("bits", 2))
        if c["op"] == "append":
            layout = kv.ROPE_HALF if c["layout"] == "half" else kv.ROPE_INTERLEAVED
            s["rope"] = kv.make_rope(s["inv_freq"], layout=layout, eps=1e-6)
            s["workspace"] = kv.alloc_workspace(s["cfg"], 0, 0)
        else:
            s["workspace"] = kv.alloc_prefix_workspace(s["cfg"], c["batch"], s["prefix_table"].shape[0])
        if c["op"] == "append" and c["cache"] == "packed":
            s["pool"] = kv.alloc_pool(s["cfg"], s["n_pool"])
    if c["op"] == "append":
        more = dict(cu_tokens=s["cu_tokens"], rope_pos=s["rope_pos"], q_weight=s["q_weight"], k_weight=s["k_weight"])
        if c["cache"] == "bf16":
            kv.append_rope_bf16(s["cfg"], s["rope"], s["pool"], s["block_table"], s["pos"], s["q"], s["k"], s["v"],
                                s["q_out"], s["workspace"], **more)
            return s["q_out"], s["pool"]
        kv.append_rope(s["cfg"], s["rope"], s["pool"], s["staging"], s["block_table"], s["pos"], s["q"], s["k"], s["v"],
                       s["q_out"], s["workspace"], **more)
        return s["q_out"], s["staging"]
    if c["cache"] == "bf16":
        kv.prefix_attn_bf16(s["cfg"], s["q"], s["pool"], s["prefix_table"], s["prefix_lens"], s["block_table"],
                            s["seq_lens"], s["out"], s["workspace"])
    else:
        kv.prefix_attn(s["cfg"], s["q"], s["pool"], s["staging"], s["prefix_table"], s["prefix_lens"], s["block_table"],
                       s["seq_lens"], s["out"], s["workspace"])
    return s["out"]


def _token_places(s):
    """Sequence and index after the cached tokens of each row."""
    T = s["q"].shape[0]
    at = torch.arange(T, device="cuda")
    if s["cu_tokens"] is None:
        return at, torch.zeros_like(at)
    seq = (at[:, None] >= s["cu_tokens"][None, 1:]).sum(1)
    return seq, at - s["cu_tokens"][seq]


def _normed(x, weight):
    x = x.float()
    if weight is None:
        return x
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * weight.float()


def _rotated(x, cos, sin, rotary, layout):
    cos, sin = cos[:, None], sin[:, None]
    if layout == "half":
        a, b = x[..., :rotary // 2], x[..., rotary // 2:rotary]
        return torch.cat([a * cos - b * sin, b * cos + a * sin, x[..., rotary:]], -1)
    a, b = x[..., 0:rotary:2], x[..., 1:rotary:2]
    pairs = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([pairs, x[..., rotary:]], -1)


def _plain_append(s):
    c = s["case"]
    seq, i = _token_places(s)
    angle = (s["rope_pos"][seq] + i).double()[:, None] * s["freq"]   # 32 bits lose the angles of far positions
    cos, sin = angle.cos().float(), angle.sin().float()
    q = _rotated(_normed(s["q"], s["q_weight"]), cos, sin, c["rotary"], c["layout"])
    k = _rotated(_normed(s["k"], s["k_weight"]), cos, sin, c["rotary"], c["layout"])
    s["q_out"].copy_(q.to(torch.bfloat16))
    at = s["pos"][seq] + i
    row = (at % c["block"])[:, None]
    heads = torch.arange(c["n_kv"], device="cuda")[None]
    if c["cache"] == "bf16":
        where, into = s["block_table"][seq, at // c["block"]][:, None], s["pool"]
    else:
        where, into = seq[:, None], s["staging"]
    into[where, heads, 0, row] = k.to(torch.bfloat16)
    into[where, heads, 1, row] = s["v"]
    return s["q_out"], into


def _hadamard(dtype):
    h = torch.ones(1, 1, dtype=dtype, device="cuda")
    for _ in range(7):
        h = torch.cat([torch.cat([h, h], 1), torch.cat([h, -h], 1)], 0)
    return h


def _values(s, table):
    """fp32 (K, V) in the rotated space, each [*table, n_kv, B, 128], of the packed blocks of a table."""
    c = s["case"]
    B, bits, n_kv = c["block"], c["bits"], c["n_kv"]
    x = 16 * bits * B
    block = s["pool"].view(s["n_pool"], n_kv, 2, -1)[table.long()]
    half = block[..., x:].contiguous().view(torch.float16).float()
    step, zero = (half[..., 4 * B * k:4 * B * (k + 1)].unflatten(-1, (4, B)).transpose(-1, -2) for k in (0, 1))
    step, zero = (y.repeat_interleave(32, -1) for y in (step, zero))
    factor = half[..., 8 * B:9 * B, None] * half[..., None, 9 * B:]
    words = block[..., :x].contiguous().view(torch.int32)
    codes = []
    for kind in (0, 1):
        word, bit, high_word, high_bit = s["places"][kind]
        mine = words[..., kind, :]
        code = (mine[..., word] >> bit) & (15 if bits == 4 else 3)
        if bits == 3:
            code = code | (((mine[..., high_word] >> high_bit) & 1) << 2)
        codes.append(code)
    y = (torch.stack(codes, -3).float() * step + zero) * factor
    return y[..., 0, :, :], y[..., 1, :, :]


def _masked(scores, shown):
    """The scores, -inf where a token is not shown to the query."""
    return torch.where(shown, scores, torch.full_like(scores, -math.inf))


def _plain_prefix(s):
    c = s["case"]
    b, n_kv, B = c["batch"], c["n_kv"], c["block"]
    G = c["n_q"] // n_kv
    q = s["q"].float().view(b, n_kv, G, D) / math.sqrt(D)
    packed = c["cache"] == "packed"
    if packed:
        H = s["hadamard"]
        qc = (q * s["signs"]) @ H
        kp, vp = _values(s, s["prefix_table"])
        ko, vo = _values(s, s["block_table"])
        inside = s["seq_lens"] // B * B      # own tokens in complete blocks; the others are raw
    else:
        qc = q
        kp, vp = s["pool"][s["prefix_table"].long()].float().unbind(2)
        ko, vo = s["pool"][s["block_table"].long()].float().unbind(3)
        inside = s["seq_lens"]
    kp, vp = (y.transpose(0, 1).flatten(1, 2) for y in (kp, vp))                   # [n_kv][tokens][128]
    ko, vo = (y.transpose(1, 2).flatten(2, 3) for y in (ko, vo))                   # [b][n_kv][tokens][128]
    sp = (qc.transpose(0, 1).flatten(1, 2) @ kp.transpose(1, 2)).unflatten(1, (b, G)).transpose(0, 1)
    so = qc @ ko.transpose(2, 3)
    at = torch.arange(sp.shape[-1], device="cuda")
    sp = _masked(sp, (at < s["prefix_lens"][:, None])[:, None, None])
    at = torch.arange(so.shape[-1], device="cuda")
    so = _masked(so, (at < inside[:, None])[:, None, None])
    all_scores = [sp, so]
    if packed:
        kt, vt = s["staging"].float().unbind(2)
        at = torch.arange(B, device="cuda")
        st = _masked(q @ kt.transpose(2, 3), (at < (s["seq_lens"] - inside)[:, None])[:, None, None])
        all_scores.append(st)
    top = torch.stack([y.amax(-1) for y in all_scores]).amax(0)[..., None]
    weights = [torch.exp(y - top) for y in all_scores]
    total = torch.stack([w.sum(-1) for w in weights]).sum(0)[..., None]
    wp = weights[0].transpose(0, 1).flatten(1, 2)
    acc = (wp @ vp).unflatten(1, (b, G)).transpose(0, 1) + weights[1] @ vo
    if packed:
        acc = (acc @ H) * s["signs"] + weights[2] @ vt
    s["out"].copy_((acc / total).flatten(1, 2).to(torch.bfloat16))
    return s["out"]


# ------------------------------------------------------------------ what a pass cannot do without

def work(c):
    n_q, n_kv, batch = c["n_q"], c["n_kv"], c["batch"]
    if c["op"] == "append":
        T = batch * c["tokens"]
        return {"bytes": 2.0 * T * (n_q + 2 * n_kv) * D * 2, "flops": T * (n_q + n_kv) * D * 6.0}
    shared = c["prefix"] * max(0, batch - 1) if batch > 2 else c["prefix"] * batch
    ctx = 0.75 * c["ctx"]
    per = n_kv * 2 * (256.0 if c["cache"] == "bf16" else _block_bytes(c["block"], c["bits"]) / c["block"])
    return {"bytes": (c["prefix"] + batch * ctx) * per + batch * n_q * D * 4.0,
            "flops": 4.0 * n_q * D * (shared + batch * ctx)}


# ------------------------------------------------------------------ the definition, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return (_exact_append if case["op"] == "append" else _exact_prefix)(case, s)


def _exact_append(c, s):
    """Each pair as a complex number, turned by exp(i position frequency)."""
    n_q, n_kv, B, T = c["n_q"], c["n_kv"], c["block"], s["q"].shape[0]
    pos, far = s["pos"].tolist(), s["rope_pos"].tolist()
    cu = list(range(T + 1)) if s["cu_tokens"] is None else s["cu_tokens"].tolist()
    at = torch.cat([torch.arange(pos[b], pos[b] + cu[b + 1] - cu[b], dtype=torch.int64) for b in range(c["batch"])]).cuda()
    turn = torch.cat([torch.arange(far[b], far[b] + cu[b + 1] - cu[b], dtype=torch.float64) for b in range(c["batch"])]).cuda()
    unit = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), turn[:, None] * s["freq"])
    done = []
    for x, weight in ((s["q"], s["q_weight"]), (s["k"], s["k_weight"])):
        x = x.double()
        if weight is not None:
            x = x / (x.square().sum(2, keepdim=True) / D + 1e-6).sqrt() * weight.double()
        r = c["rotary"]
        if c["layout"] == "half":
            z = torch.complex(x[:, :, :r // 2].contiguous(), x[:, :, r // 2:r].contiguous()) * unit[:, None]
            x[:, :, :r // 2], x[:, :, r // 2:r] = z.real, z.imag
        else:
            z = torch.complex(x[:, :, :r:2].contiguous(), x[:, :, 1:r:2].contiguous()) * unit[:, None]
            x[:, :, :r:2], x[:, :, 1:r:2] = z.real, z.imag
        done.append(x)
    into = (s["pool"] if c["cache"] == "bf16" else s["staging"]).double()
    table = s["block_table"].long().cpu()
    for b in range(c["batch"]):
        rows = slice(cu[b], cu[b + 1])
        t = at[rows]
        where = table[b].cuda()[t // B] if c["cache"] == "bf16" else torch.full_like(t, b)
        into[where, :, 0, t % B] = done[1][rows]
        into[where, :, 1, t % B] = s["v"][rows].double()
    return done[0], into


def _exact_codes(words, kind, B, bits):
    """[..., B, 128] codes from the 32-bit words [..., (B / 32) 8 4 (4 bits)] of a head-block's records: each
    word taken apart into its fields, and the fields' axes put in the order of tokens and channels."""
    n = words.shape[0]
    bit = (words.view(n, -1)[:, :, None] >> torch.arange(32, device="cuda")) & 1        # [n][words][32]
    if bits == 3:
        rec = bit.view(n, B // 32, 8, 4, 12, 32)
        low, high = rec[..., :8, :].flatten(1), rec[..., 8:, :].flatten(1)
        # the high bit of word w's field j in half h: word w / 2, bit 8 (w % 2) + j + 16 h
        high = high.view(n, B // 32, 8, 4, 4, 2, 2, 8).transpose(-3, -2).reshape(n, B // 32, 8, 4, 8, 2, 8)
        code = low.view(n, B // 32, 8, 4, 8, 2, 8, 2)
        code = code[..., 0] + 2 * code[..., 1] + 4 * high                                # [n][sb][a][b][w][h][j]
        bits = 2
    else:
        code = (bit.view(n, B // 32, 8, 4, 4 * bits, 2, 16 // bits, bits) << torch.arange(bits, device="cuda")).sum(-1)
    if bits == 2 and kind == 0:      # w = (i, g / 2), j = (g % 2, e / 2), h = e % 2
        code = code.view(n, B // 32, 8, 4, 4, 2, 2, 2, 4).permute(0, 1, 2, 4, 5, 7, 3, 8, 6)
    elif bits == 2:                  # w = (g, f / 2), j = (d / 4, d % 4 / 2, f % 2), h = d % 2
        code = code.view(n, B // 32, 8, 4, 4, 2, 2, 2, 2, 2).permute(0, 1, 3, 7, 8, 6, 4, 2, 5, 9)
    elif kind == 0:                  # w = (i, g), j = e / 2, h = e % 2
        code = code.view(n, B // 32, 8, 4, 4, 4, 2, 4).permute(0, 1, 2, 4, 5, 3, 7, 6)
    else:                            # w = (g, f), j = d / 2, h = d % 2
        code = code.view(n, B // 32, 8, 4, 4, 4, 2, 4).permute(0, 1, 3, 7, 6, 4, 2, 5)
    return code.reshape(n, B, D)


def _exact_head(c, s, ids, h):
    """fp64 (K, V), each [len(ids) B][128], of kv head h of the blocks `ids`, in the space of the query."""
    B = c["block"]
    if c["cache"] == "bf16":
        mine = s["pool"][ids, h].double()
        return mine[:, 0].reshape(-1, D), mine[:, 1].reshape(-1, D)
    bits, n = c["bits"], len(ids)
    raw = s["pool"].view(s["n_pool"], c["n_kv"], 2, -1)[ids, h]
    back = _hadamard(torch.float64) / math.sqrt(D)
    both = []
    for kind in (0, 1):
        mine = raw[:, kind].contiguous()
        code = _exact_codes(mine[:, :16 * bits * B].contiguous().view(torch.int32), kind, B, bits).double()
        rest = mine[:, 16 * bits * B:].contiguous().view(torch.float16).double()
        per = [rest[:, 4 * B * k:4 * B * k + 4 * B].view(n, 4, B).permute(0, 2, 1)[..., None] for k in (0, 1)]
        val = (code.view(n, B, 4, 32) * per[0] + per[1]).view(n, B, D)
        val = val * rest[:, 8 * B:9 * B, None] * rest[:, None, 9 * B:]
        both.append((val.view(-1, D) @ back) * s["signs"].double())
    return both


def _exact_prefix(c, s):
    batch, n_kv, B = c["batch"], c["n_kv"], c["block"]
    G = c["n_q"] // n_kv
    shared, lens = s["prefix_lens"].tolist(), s["seq_lens"].tolist()
    out = torch.zeros(batch, c["n_q"], D, dtype=torch.float64, device="cuda")
    for h in range(n_kv):
        kp, vp = _exact_head(c, s, s["prefix_table"].long(), h)
        ko, vo = _exact_head(c, s, s["block_table"].long().view(-1), h)
        ko, vo = ko.view(batch, -1, D), vo.view(batch, -1, D)
        for b in range(batch):
            whole = lens[b] if c["cache"] == "bf16" else lens[b] // B * B
            k, v = [kp[:shared[b]], ko[b, :whole]], [vp[:shared[b]], vo[b, :whole]]
            if c["cache"] == "packed":
                k.append(s["staging"][b, h, 0, :lens[b] - whole].double())
                v.append(s["staging"][b, h, 1, :lens[b] - whole].double())
            k, v = torch.cat(k), torch.cat(v)
            w = torch.softmax(s["q"][b, h * G:(h + 1) * G].double() @ k.T / math.sqrt(D), -1)
            out[b, h * G:(h + 1) * G] = w @ v
    return out
