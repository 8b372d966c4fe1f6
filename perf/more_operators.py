"""Long generations over the paged caches, as cases to be measured: several drafted
tokens verified in one pass, attention weights kept along with a decode step, and a
cache cut down to a budget by those weights.

Three kinds of case (``op``), each for both caches (``cache``: "bf16" pages, or
"packed" head-blocks of 2-, 3- or 4-bit codes with a bf16 staging buffer):

tree     the queries of a sequence's drafted tokens (a tree; draft i is shown to
         query row r where mask[b][r] has bit i) over the cached tokens, which all
         rows see, and the drafts' own keys and values, which are not cached yet.
weights  decode attention; beside the output, decay * weights + the softmax weight
         of each cached token, summed over the query heads of its kv head.
evict    a sequence longer than `budget` keeps its last `recent` tokens and, of the
         others, those with the greatest weights (ties: the lowest index), each kv
         head its own; what is kept goes, in order, to other pages with its weights.
         Packed: whole blocks, by the sum of their tokens' weights (rounded to 32
         bits); the incomplete block stays in staging.

``own`` selects the plain torch form (False) or the package's kernels (True).
"""
import math

import numpy as np
import torch

own = False

D = 128


# ------------------------------------------------------------------ cases

def _tree(name, cache, batch, drafts, ctx, n_q, n_kv, block, bits, shape, query="bf16"):
    return dict(name=name, op="tree", cache=cache, batch=batch, drafts=drafts, ctx=ctx, n_q=n_q, n_kv=n_kv, block=block,
                bits=bits, shape=shape, query=query)


def _weights(name, cache, batch, ctx, n_q, n_kv, block, bits, decay, query="bf16"):
    return dict(name=name, op="weights", cache=cache, batch=batch, ctx=ctx, n_q=n_q, n_kv=n_kv, block=block, bits=bits,
                decay=decay, query=query)


def _evict(name, cache, batch, ctx, budget, recent, n_kv, block, bits):
    return dict(name=name, op="evict", cache=cache, batch=batch, ctx=ctx, budget=budget, recent=recent, n_q=n_kv,
                n_kv=n_kv, block=block, bits=bits)


def listed():
    return [
        # one user, a few drafts of a small draft model: the latency of a call
        _tree("tree-bf16-1x8-1k", "bf16", 1, 8, 1000, 32, 8, 32, 2, "tree"),
        # a batch of long sequences with trees of an odd size, not all of them full
        _tree("tree-bf16-32x33-8k", "bf16", 32, 33, 8192, 32, 8, 64, 2, "ragged"),
        # the same two uses over the packed cache: a few users with a chain of drafts, and a batch
        _tree("tree-2bit-3x12-1500", "packed", 3, 12, 1500, 40, 10, 32, 2, "chain"),
        _tree("tree-4bit-48x16-8k", "packed", 48, 16, 8192, 32, 8, 64, 4, "tree"),
        # a decode step of two users that keeps its weights
        _weights("weights-bf16-2x1k", "bf16", 2, 1000, 32, 8, 32, 2, 1.0),
        # a batch of long sequences, older steps counting for less
        _weights("weights-bf16-32x8k", "bf16", 32, 8192, 32, 8, 64, 2, 0.97),
        # the same over the packed cache: a few odd sequences, and the benchmark's batch and length
        _weights("weights-2bit-5x1500", "packed", 5, 1500, 40, 10, 32, 2, 1.0),
        _weights("weights-2bit-64x8k", "packed", 64, 8192, 32, 8, 64, 2, 1.0),
        # two users' short caches cut to a quarter
        _evict("evict-bf16-2x1k", "bf16", 2, 1000, 250, 33, 8, 32, 2),
        # a batch of long sequences cut to a budget
        _evict("evict-bf16-32x8k", "bf16", 32, 8192, 2048, 256, 8, 64, 2),
        # packed blocks: a few odd sequences, and a batch of the longest
        _evict("evict-2bit-5x1500", "packed", 5, 1500, 512, 64, 10, 32, 2),
        _evict("evict-2bit-64x16k", "packed", 64, 16384, 4096, 512, 8, 64, 2),
    ]


def _log(rng, lo, hi):
    """A whole number from lo to hi, spread over its logarithm."""
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op, cache = rng.choice(["tree", "weights", "evict"]), rng.choice(["bf16", "packed"])
    n_kv, group = rng.choice([1, 2, 3, 4, 8, 10]), rng.choice([1, 2, 3, 4])
    block, bits, query = rng.choice([32, 64]), rng.choice([2, 3, 4]), rng.choice(["bf16", "bf16", "fp32"])
    batch = _log(rng, 1, 64)
    if op == "tree":
        drafts = _log(rng, 1, 96)
        ctx = _log(rng, 1, max(1, min(16384, 2000000 // (batch * n_kv), 250000000 // (batch * drafts * n_kv * group))))
        c = _tree("", cache, batch, drafts, ctx, n_kv * group, n_kv, block, bits,
                  rng.choice(["tree", "chain", "ragged"]), query)
    elif op == "weights":
        ctx = _log(rng, 1, min(32768, (4000000 if cache == "packed" else 2000000) // (batch * n_kv)))
        c = _weights("", cache, batch, ctx, n_kv * group, n_kv, block, bits, rng.choice([1.0, 0.97, 0.5]), query)
    else:
        ctx = _log(rng, 1, min(32768, (8000000 if cache == "packed" else 2000000) // (batch * n_kv)))
        budget = _log(rng, 1, max(1, min(2 * ctx, 600000 // (batch * n_kv))))
        recent = rng.randint(0, budget)
        if cache == "packed":
            budget = -(-budget // block) * block
            recent = recent // block * block
        c = _evict("", cache, batch, ctx, budget, recent, n_kv, block, bits)
    del c["name"]
    return c


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    r = np.random.RandomState(int(seed) % (1 << 31))
    c = case
    batch, n_kv, B, ctx = c["batch"], c["n_kv"], c["block"], c["ctx"]
    lens = r.randint(max(1, ctx // 2), ctx + 1, batch)
    if batch > 3:
        lens[r.randint(batch)] = 0          # a sequence that has just begun
    nb = -(-ctx // B)
    new_nb = c["budget"] // B + 1 if c["op"] == "evict" else 0
    n_pool = batch * (nb + new_nb) + 2
    pages = r.permutation(n_pool)
    s = dict(case=c, seq_lens=_ints(lens), n_pool=n_pool, nb=nb, new_nb=new_nb,
             block_table=_ints(pages[:batch * nb].reshape(batch, nb)),
             new_table=_ints(pages[batch * nb:batch * (nb + new_nb)].reshape(batch, new_nb)))
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
    if c["op"] == "tree":
        _prepare_tree(c, s, g, r)
    elif c["op"] == "weights":
        s["q"] = _queries(c, (batch, c["n_q"], D), g)
        s["out"] = torch.zeros(batch, c["n_q"], D, dtype=torch.bfloat16, device="cuda")
        s["weights"] = _worth(c, s, g)
        s["new_weights"] = torch.zeros_like(s["weights"])
    else:
        s["weights"] = _worth(c, s, g)
        s["new_weights"] = torch.zeros(batch, n_kv, new_nb * B, device="cuda")
        s["new_lens"] = torch.zeros(batch, dtype=torch.int32, device="cuda")
        each = c["budget"] if c["cache"] == "bf16" else c["budget"] // B
        s["kept"] = torch.zeros(batch, n_kv, each, dtype=torch.int32, device="cuda")
    return s


def _ints(values):
    return torch.tensor(np.asarray(values), dtype=torch.int32, device="cuda")


def _queries(c, shape, g):
    q = 2 * torch.randn(*shape, generator=g, device="cuda")   # scores of a few units
    return q if c["query"] == "fp32" else q.to(torch.bfloat16)


def _worth(c, s, g):
    """Attention weights as some hundred decode steps leave them: a heavy tail, and tokens that nothing has looked at."""
    shape = (c["batch"], c["n_kv"], s["nb"] * c["block"])
    w = torch.exp(1.5 * torch.randn(*shape, generator=g, device="cuda")) * (300.0 / c["ctx"])
    w *= torch.rand(*shape, generator=g, device="cuda") > 0.1
    return w * (torch.arange(shape[2], device="cuda") < s["seq_lens"][:, None])[:, None]


def _prepare_tree(c, s, g, r):
    batch, T, n_q, n_kv = c["batch"], c["drafts"], c["n_q"], c["n_kv"]
    shown = np.zeros((batch, T, T), bool)
    for b in range(batch):
        for i in range(T):
            # a branch goes on from a recent draft, or begins at the last cached token
            parent = i - 1 if c["shape"] == "chain" else max(-1, i - 1 - min(r.geometric(0.4) - 1, 7))
            if parent >= 0:
                shown[b, i] = shown[b, parent]
            shown[b, i, i] = True
    if c["shape"] == "tree" and T > 4:
        shown[r.randint(batch), r.randint(T)] = False        # a row that sees the cached tokens alone
    words = -(-T // 32)
    bits = np.zeros((batch, T, words * 32), np.uint64)
    bits[..., :T] = shown
    mask = (bits.reshape(batch, T, words, 32) << np.arange(32, dtype=np.uint64)).sum(-1).astype(np.uint32)
    rows = torch.randn(batch, T, 2 * n_kv * D, generator=g, device="cuda").to(torch.bfloat16)
    s["shown"] = torch.from_numpy(shown).cuda()
    s["mask"] = torch.from_numpy(mask.view(np.int32)).cuda()
    s["k"] = rows[..., :n_kv * D].unflatten(-1, (n_kv, D))   # columns of one projection's rows
    s["v"] = rows[..., n_kv * D:].unflatten(-1, (n_kv, D))
    s["draft_lens"] = _ints(r.randint(1, T + 1, batch)) if c["shape"] == "ragged" else None
    s["q"] = _queries(c, (batch, T, n_q, D), g)
    s["out"] = torch.zeros(batch, T, n_q, D, dtype=torch.bfloat16, device="cuda")


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
    op = state["case"]["op"]
    if own:
        return {"tree": _own_tree, "weights": _own_weights, "evict": _own_evict}[op](state)
    return {"tree": _plain_tree, "weights": _plain_weights, "evict": _plain_evict}[op](state)


def _config(kv, s):
    c = s["case"]   # what a program sets up once for its model and batch
    s["cfg"] = kv.make_config(c["n_q"], c["n_kv"], c["block"], 2, s.get("sign_bits", [0, 0, 0, 0]), bits=c["bits"])
    if c["op"] == "tree":
        s["workspace"] = kv.alloc_tree_workspace(s["cfg"], c["batch"], c["drafts"], s["nb"])
    elif c["op"] == "weights":
        s["workspace"] = kv.alloc_weights_workspace(s["cfg"], c["batch"], s["nb"])
    else:
        s["workspace"] = kv.alloc_workspace(s["cfg"], 0, 0)


def _own_tree(s):
    import bit_kv_cache_08_gb300 as kv
    if "cfg" not in s:
        _config(kv, s)
    rest = (s["block_table"], s["seq_lens"], s["k"], s["v"], s["mask"], s["out"], s["workspace"])
    if s["case"]["cache"] == "bf16":
        kv.tree_attn_bf16(s["cfg"], s["q"], s["pool"], *rest, draft_lens=s["draft_lens"])
    else:
        kv.tree_attn(s["cfg"], s["q"], s["pool"], s["staging"], *rest, draft_lens=s["draft_lens"])
    return s["out"]


def _own_weights(s):
    import bit_kv_cache_08_gb300 as kv
    if "cfg" not in s:
        _config(kv, s)
    rest = (s["block_table"], s["seq_lens"], s["out"], s["new_weights"], s["workspace"])
    more = dict(weights_in=s["weights"], decay=s["case"]["decay"])
    if s["case"]["cache"] == "bf16":
        kv.decode_attn_weights_bf16(s["cfg"], s["q"], s["pool"], *rest, **more)
    else:
        kv.decode_attn_weights(s["cfg"], s["q"], s["pool"], s["staging"], *rest, **more)
    return s["out"], s["new_weights"]


def _own_evict(s):
    import bit_kv_cache_08_gb300 as kv
    c = s["case"]
    if "cfg" not in s:
        _config(kv, s)
    call = kv.evict_bf16 if c["cache"] == "bf16" else kv.evict
    call(s["cfg"], s["pool"], s["block_table"], s["seq_lens"], s["weights"], s["new_table"], s["new_lens"],
         s["new_weights"], s["kept"], s["workspace"], budget=c["budget"], recent=c["recent"])
    return s["new_lens"], s["kept"], s["new_weights"], _moved(s)


def _moved(s):
    """The pages that an eviction writes to: rows of bf16, or the blocks' 32-bit words (moved as they are)."""
    if s["case"]["cache"] == "bf16":
        return s["pool"]
    return s["pool"].view(torch.int32)


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
    found = []
    for kind in (0, 1):
        word, bit, high_word, high_bit = s["places"][kind]
        mine = words[..., kind, :]
        code = (mine[..., word] >> bit) & (15 if bits == 4 else 3)
        if bits == 3:
            code = code | (((mine[..., high_word] >> high_bit) & 1) << 2)
        found.append((code.float() * step[..., kind, :, :] + zero[..., kind, :, :]) * factor[..., kind, :, :])
    return found


def _masked(scores, shown):
    """The scores, -inf where a token is not shown to the query."""
    return torch.where(shown, scores, torch.full_like(scores, -math.inf))


def _cached(s, q):
    """Query rows q [batch][n_kv][rows][128] (times the scale) over the cached tokens: their scores
    [batch][n_kv][rows][tokens], -inf behind the end, and the function that weighs the values."""
    c = s["case"]
    B, lens = c["block"], s["seq_lens"][:, None, None, None]
    if c["cache"] == "bf16":
        k, v = (y.transpose(1, 2).flatten(2, 3) for y in s["pool"][s["block_table"].long()].float().unbind(3))
        at = torch.arange(k.shape[2], device="cuda")
        return _masked(q @ k.transpose(2, 3), at < lens), lambda w: w @ v
    H = s["hadamard"]
    k, v = (y.transpose(1, 2).flatten(2, 3) for y in _values(s, s["block_table"]))
    kt, vt = s["staging"].float().unbind(2)
    at = torch.arange(k.shape[2], device="cuda")
    inside = lens // B * B                       # tokens in complete blocks; the others are raw
    raw = (at - inside).clamp(0, B - 1)
    scores = ((q * s["signs"]) @ H) @ k.transpose(2, 3)
    tail = (q @ kt.transpose(2, 3)).gather(-1, raw.expand(*q.shape[:3], -1))
    scores = _masked(torch.where(at < inside, scores, tail), at < lens)

    def weigh(w):
        there = (inside + torch.arange(B, device="cuda")).expand(*w.shape[:3], -1)
        last = torch.where(there < lens, w.gather(-1, there.clamp(max=w.shape[-1] - 1)), torch.zeros_like(there, dtype=w.dtype))
        return ((torch.where(at < inside, w, torch.zeros_like(w)) @ v) @ H) * s["signs"] + last @ vt

    return scores, weigh


def _finite(top):
    return torch.where(torch.isinf(top), torch.zeros_like(top), top)


def _plain_tree(s):
    c = s["case"]
    batch, T, n_kv = c["batch"], c["drafts"], c["n_kv"]
    G = c["n_q"] // n_kv
    q = (s["q"].float() / math.sqrt(D)).view(batch, T, n_kv, G, D).permute(0, 2, 1, 3, 4).flatten(2, 3)
    scores, weigh = _cached(s, q)
    k, v = (y.float().transpose(1, 2) for y in (s["k"], s["v"]))                  # [batch][n_kv][T][128]
    rows = torch.arange(T, device="cuda")
    lens = torch.full((batch,), T, device="cuda") if s["draft_lens"] is None else s["draft_lens"]
    shown = s["shown"] & (rows < lens[:, None])[:, None]
    drafted = _masked(q @ k.transpose(2, 3), shown.repeat_interleave(G, 1)[:, None])
    top = _finite(torch.maximum(scores.amax(-1), drafted.amax(-1))[..., None])
    w, wd = torch.exp(scores - top), torch.exp(drafted - top)
    total = (w.sum(-1) + wd.sum(-1))[..., None]
    out = (weigh(w) + wd @ v) / torch.where(total > 0, total, torch.ones_like(total))
    out = out.unflatten(2, (T, G)).permute(0, 2, 1, 3, 4).flatten(2, 3).to(torch.bfloat16)
    s["out"].copy_(torch.where((rows < lens[:, None])[..., None, None], out, s["out"]))
    return s["out"]


def _plain_weights(s):
    c = s["case"]
    batch, n_kv = c["batch"], c["n_kv"]
    scores, weigh = _cached(s, s["q"].float().view(batch, n_kv, -1, D) / math.sqrt(D))
    w = torch.exp(scores - _finite(scores.amax(-1, keepdim=True)))
    total = w.sum(-1, keepdim=True)
    w = w / torch.where(total > 0, total, torch.ones_like(total))
    s["out"].copy_(weigh(w).flatten(1, 2).to(torch.bfloat16))
    there = (torch.arange(w.shape[-1], device="cuda") < s["seq_lens"][:, None])[:, None]
    s["new_weights"].copy_(torch.where(there, c["decay"] * s["weights"] + w.sum(2), s["new_weights"]))
    return s["out"], s["new_weights"]


def _plain_evict(s):
    c = s["case"]
    batch, n_kv, B = c["batch"], c["n_kv"], c["block"]
    lens = s["seq_lens"].long()
    packed = c["cache"] == "packed"
    worth, unit = s["weights"], 1
    if packed:    # whole blocks, by the sum of their tokens' weights
        worth, unit = worth.double().unflatten(-1, (-1, B)).sum(-1).float(), B
    have, budget, recent = (lens // unit)[:, None, None], c["budget"] // unit, c["recent"] // unit
    at = torch.arange(worth.shape[-1], device="cuda")
    key = torch.where(at >= have - recent, torch.full_like(worth, math.inf), worth)
    key = torch.where(at < have, key, torch.full_like(worth, -1.0))
    order = key.sort(dim=-1, descending=True, stable=True).indices[..., :budget].sort(-1).values
    if order.shape[-1] < budget:
        order = torch.nn.functional.pad(order, (0, budget - order.shape[-1]), value=worth.shape[-1])
    valid = order < have
    s["kept"].copy_(torch.where(valid, order, torch.full_like(order, -1)))
    order = torch.where(valid, order, torch.zeros_like(order))
    tail = lens % unit
    s["new_lens"].copy_((have[:, 0, 0].clamp(max=budget) * unit + tail).to(torch.int32))
    b = torch.arange(batch, device="cuda")[:, None, None]
    h = torch.arange(n_kv, device="cuda")[None, :, None]
    i = torch.arange(budget, device="cuda")
    if packed:
        blocks = s["pool"].view(s["n_pool"], n_kv, -1)
        to = s["new_table"].long()[b, i.expand(batch, n_kv, -1)]
        source = torch.where(valid, s["block_table"].long()[b, order], to)
        blocks[to, h] = blocks[source, h]
    else:
        to, row = s["new_table"].long()[b, (i // B).expand(batch, n_kv, -1)], i % B
        source = torch.where(valid, s["block_table"].long()[b, order // B], to)
        s["pool"][to, h, :, row] = s["pool"][source, h, :, torch.where(valid, order % B, row)]
    # the kept tokens' weights, those of the incomplete block, and zeros behind
    col = torch.arange(s["new_weights"].shape[-1], device="cuda").expand(batch, n_kv, -1)
    size = have.clamp(max=budget) * unit
    slot = (col // unit).clamp(max=budget - 1)
    source = order.gather(-1, slot) * unit + col % unit
    source = torch.where(col < size, source, have * unit + col - size).clamp(0, s["weights"].shape[-1] - 1)
    taken = s["weights"].gather(-1, source)
    s["new_weights"].copy_(torch.where(col < size + tail[:, None, None], taken, torch.zeros_like(taken)))
    return s["new_lens"], s["kept"], s["new_weights"], _moved(s)


# ------------------------------------------------------------------ what a pass cannot do without

def work(c):
    batch, n_q, n_kv, B = c["batch"], c["n_q"], c["n_kv"], c["block"]
    tokens = batch * 0.75 * c["ctx"]
    per = n_kv * 2 * (256.0 if c["cache"] == "bf16" else _block_bytes(B, c["bits"]) / B)   # bytes of a cached token
    query = 4.0 if c.get("query") == "fp32" else 2.0
    if c["op"] == "tree":
        rows = batch * c["drafts"]
        return {"bytes": tokens * per + rows * (n_q * D * (2.0 + query) + 2 * n_kv * D * 2.0),
                "flops": 4.0 * D * n_q * c["drafts"] * tokens}
    if c["op"] == "weights":
        return {"bytes": tokens * (per + n_kv * 8.0) + batch * n_q * D * (2.0 + query), "flops": 4.0 * D * n_q * tokens}
    kept = batch * min(0.75 * c["ctx"], c["budget"])
    return {"bytes": tokens * n_kv * 4.0 + kept * (2 * per + n_kv * 4.0), "flops": 0.0}


# ------------------------------------------------------------------ the definition, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"tree": _exact_tree, "weights": _exact_weights, "evict": _exact_evict}[case["op"]](case, s)


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


def _exact_tokens(c, s, b, h):
    """fp64 (K, V), each [seq_lens[b]][128], of kv head h of sequence b, in the space of the query."""
    B, L = c["block"], int(s["seq_lens"][b])
    ids = s["block_table"][b].long()
    if c["cache"] == "bf16":
        mine = s["pool"][ids[:-(-L // B)], h].double()
        return mine[:, 0].reshape(-1, D)[:L], mine[:, 1].reshape(-1, D)[:L]
    bits, n = c["bits"], L // B
    raw = s["pool"].view(s["n_pool"], c["n_kv"], 2, -1)[ids[:n], h]
    back = _hadamard(torch.float64) / math.sqrt(D)
    both = []
    for kind in (0, 1):
        rows = s["staging"][b, h, kind, :L - n * B].double()
        if n:
            mine = raw[:, kind].contiguous()
            code = _exact_codes(mine[:, :16 * bits * B].contiguous().view(torch.int32), kind, B, bits).double()
            rest = mine[:, 16 * bits * B:].contiguous().view(torch.float16).double()
            per = [rest[:, 4 * B * k:4 * B * k + 4 * B].view(n, 4, B).permute(0, 2, 1)[..., None] for k in (0, 1)]
            val = (code.view(n, B, 4, 32) * per[0] + per[1]).view(n, B, D)
            val = val * rest[:, 8 * B:9 * B, None] * rest[:, None, 9 * B:]
            rows = torch.cat([(val.view(-1, D) @ back) * s["signs"].double(), rows])
        both.append(rows)
    return both


def _exact_tree(c, s):
    n_kv, T = c["n_kv"], c["drafts"]
    G = c["n_q"] // n_kv
    out = s["out"].double()
    lens = [T] * c["batch"] if s["draft_lens"] is None else s["draft_lens"].tolist()
    for b in range(c["batch"]):
        n = lens[b]
        for h in range(n_kv):
            k, v = _exact_tokens(c, s, b, h)
            cached = k.shape[0]
            k, v = torch.cat([k, s["k"][b, :n, h].double()]), torch.cat([v, s["v"][b, :n, h].double()])
            hidden = torch.cat([torch.zeros(n, cached, dtype=torch.bool, device="cuda"), ~s["shown"][b, :n, :n]], 1)
            z = s["q"][b, :n, h * G:(h + 1) * G].double() @ k.T / math.sqrt(D)
            w = torch.softmax(z.masked_fill(hidden[:, None], -math.inf), -1).nan_to_num(0.0)   # (a row that sees nothing: 0)
            out[b, :n, h * G:(h + 1) * G] = w @ v
    return out


def _exact_weights(c, s):
    n_kv, G = c["n_kv"], c["n_q"] // c["n_kv"]
    out, new = s["out"].double(), s["new_weights"].double()
    for b in range(c["batch"]):
        L = int(s["seq_lens"][b])
        for h in range(n_kv):
            if L == 0:
                continue
            k, v = _exact_tokens(c, s, b, h)
            w = torch.softmax(s["q"][b, h * G:(h + 1) * G].double() @ k.T / math.sqrt(D), -1)
            out[b, h * G:(h + 1) * G] = w @ v
            new[b, h, :L] = c["decay"] * s["weights"][b, h, :L].double() + w.sum(0)
    return out, new


def _exact_evict(c, s):
    batch, n_kv, B = c["batch"], c["n_kv"], c["block"]
    packed = c["cache"] == "packed"
    unit = B if packed else 1
    budget, recent = c["budget"] // unit, c["recent"] // unit
    table, to = s["block_table"].cpu().numpy(), s["new_table"].cpu().numpy()
    lens, worth = s["seq_lens"].cpu().numpy(), s["weights"].cpu().numpy()
    kept = np.full((batch, n_kv, budget), -1, np.int32)
    new_lens = np.zeros(batch, np.int32)
    new_weights = np.zeros(tuple(s["new_weights"].shape))
    moves = []
    for b in range(batch):
        have, L = int(lens[b]) // unit, int(lens[b])
        size = min(have, budget)
        new_lens[b] = size * unit + L % unit
        for h in range(n_kv):
            each = worth[b, h, :have * unit].reshape(have, unit).astype(np.float64).sum(1).astype(np.float32)
            pick = np.arange(have)
            if have > budget:
                old = have - recent
                best = np.lexsort((np.arange(old), -each[:old]))[:budget - recent]
                pick = np.concatenate([np.sort(best), np.arange(old, have)])
            kept[b, h, :size] = pick
            token = (pick[:, None] * unit + np.arange(unit)).ravel()
            token = np.concatenate([token, np.arange(have * unit, L)])
            new_weights[b, h, :len(token)] = worth[b, h, token]
            i = np.arange(size)
            if packed:
                moves.append((table[b, pick], to[b, i], np.full(size, h), i, i))
            else:
                moves.append((table[b, pick // B], to[b, i // B], np.full(size, h), pick % B, i % B))
    source, target, head, row, new_row = (torch.from_numpy(np.concatenate([m[k] for m in moves]).astype(np.int64)).cuda()
                                          for k in range(5))
    if packed:
        blocks = s["pool"].view(s["n_pool"], n_kv, -1)
        blocks[target, head] = blocks[source, head]
        pages = _moved(s)
    else:
        pages = s["pool"].double()
        pages[target, head, :, new_row] = pages[source, head, :, row]
    return _ints(new_lens), _ints(kept), torch.from_numpy(new_weights).cuda(), pages
