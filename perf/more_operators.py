"""Measured cases of the 8-bit paged KV cache and its rotary positions.

The operators, as a target with an 8-bit cache runs them around its projections:

  rope    rotary positions of query and key heads (half or interleaved pairs, the whole head or its
          first dims, frequencies scaled for long contexts; inverse = the backward pass)
  append  keys and values of new tokens into a paged cache, the keys rotated on the way: bf16, or
          e4m3 with a power-of-two scale for each 64 positions of a page and KV head
  attn    attention of single tokens, or of the nodes of verified trees, over the e4m3 cache

``own`` selects between the plain forms (elementary torch operations in 32 bits, angles in 64) and the
calls of this package.  4096 hidden columns are 32 query and 8 KV heads of 128, 60 nodes a tree, 2048
positions the prefix, as in the benchmark's target.
"""
import math
import random

import torch

own = False

DEV = "cuda"
F8 = torch.float8_e4m3fn
GROUP = 64   # positions that share a scale


# ------------------------------------------------------------------------------------ cases
def listed():
    return [
        # the query and key heads of one token inside a fused q/k/v row
        dict(name="rope-1", op="rope", rows=1, heads=40, pitch=48, dim=128, rot=128, layout="half", scaling="none",
             far=4096, dtype="bf16", inverse=False),
        # 64 trees of 60 nodes, frequencies of a long-context target
        dict(name="rope-3840", op="rope", rows=3840, heads=40, pitch=48, dim=128, rot=128, layout="half",
             scaling="bands", far=131072, dtype="bf16", inverse=False),
        # a ragged batch in training: gradients, interleaved pairs, part of an odd head
        dict(name="rope-back-1537", op="rope", rows=1537, heads=13, pitch=13, dim=96, rot=64, layout="interleaved",
             scaling="ramp", far=32768, dtype="f32", inverse=True),
        # the next token of one sequence
        dict(name="append-1", op="append", batch=1, new=1, length=4000, kv=8, dim=128, rot=128, layout="half",
             scaling="none", fmt="e4m3", page=64, mix=1),
        # the next token of 64 sequences of unlike lengths
        dict(name="append-64", op="append", batch=64, new=1, length=1000, kv=8, dim=128, rot=128, layout="half",
             scaling="bands", fmt="e4m3", page=128, mix=2),
        # a long prompt into an empty cache
        dict(name="append-16384", op="append", batch=1, new=16384, length=0, kv=8, dim=128, rot=128, layout="half",
             scaling="bands", fmt="e4m3", page=256, mix=3),
        # ragged prompts behind cached ones, bf16 pages of 16, interleaved pairs of part of the head
        dict(name="append-bf16", op="append", batch=7, new=999, length=500, kv=5, dim=96, rot=64, layout="interleaved",
             scaling="linear", fmt="bf16", page=16, mix=4),
        # single token of one sequence, latency
        dict(name="attn-1", op="attn", batch=1, nodes=1, tree=False, heads=32, kv=8, length=4096, page=64, mix=0),
        # single tokens of 64 sequences of unlike lengths
        dict(name="attn-64", op="attn", batch=64, nodes=1, tree=False, heads=32, kv=8, length=8192, page=128, mix=5),
        # one long context
        dict(name="attn-long", op="attn", batch=1, nodes=1, tree=False, heads=32, kv=8, length=250000, page=256, mix=0),
        # small trees, shared keys (one KV head), ragged lengths, one sequence still empty
        dict(name="attn-tree-7", op="attn", batch=7, nodes=17, tree=True, heads=12, kv=1, length=3001, page=64, mix=6),
        # 64 trees of 60 nodes
        dict(name="attn-tree-64", op="attn", batch=64, nodes=60, tree=True, heads=32, kv=8, length=2048, page=128,
             mix=0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49))))))


def _cost(case):
    w = work(case)
    return w["bytes"] / 6.8e12 + w["flops"] / 1.7e15


SCALINGS = ["none", "linear", "base", "bands", "ramp"]


def draw(rng):
    most = {op: max(_cost(c) for c in listed() if c["op"] == op) for op in ("rope", "append", "attn")}
    while True:
        op = rng.choice(["rope", "append", "attn", "attn"])
        if op == "rope":
            dim = rng.choice([64, 80, 96, 128, 256])
            heads = _log(rng, 1, 64)
            c = dict(op=op, rows=_log(rng, 1, 16384), heads=heads, pitch=heads + rng.choice([0, 0, rng.randint(1, 16)]),
                     dim=dim, rot=rng.choice([dim, dim, 32, 2 * rng.randint(2, dim // 2)]),
                     layout=rng.choice(["half", "interleaved"]), scaling=rng.choice(SCALINGS),
                     far=_log(rng, 1, 1 << 20), dtype=rng.choice(["bf16", "bf16", "f32"]), inverse=rng.random() < 0.4)
        elif op == "append":
            dim = rng.choice([64, 96, 128, 128, 256])
            fmt = rng.choice(["e4m3", "e4m3", "bf16"])
            c = dict(op=op, batch=_log(rng, 1, 64), new=_log(rng, 1, 16384), length=rng.choice([0, _log(rng, 1, 4096)]),
                     kv=rng.randint(1, 16), dim=dim, rot=rng.choice([0, dim, dim, 32, 2 * rng.randint(2, dim // 2)]),
                     layout=rng.choice(["half", "interleaved"]), scaling=rng.choice(SCALINGS), fmt=fmt,
                     page=rng.choice([64, 128, 192, 256]) if fmt == "e4m3" else rng.choice([1, 16, 17, 64]),
                     mix=rng.randint(1, 1 << 20))
        else:
            kv = rng.choice([1, 2, 3, 4, 8, 8])
            tree = rng.random() < 0.5
            c = dict(op=op, batch=_log(rng, 1, 64), nodes=_log(rng, 1, 64) if tree else rng.choice([1, 1, 1, 2, 5]),
                     tree=tree, heads=kv * rng.choice([1, 2, 3, 4, 4, 8, 16]), kv=kv, length=_log(rng, 1, 131072),
                     page=rng.choice([64, 128, 192, 256]), mix=rng.choice([0, rng.randint(1, 1 << 20)]))
            if c["batch"] * c["length"] * c["kv"] > 1 << 22:   # at most 1 GB of cache
                continue
            if c["batch"] * c["nodes"] * c["heads"] * c["length"] > 1 << 29:   # scores of the plain form
                continue
        if _cost(c) <= most[op]:
            return c


def _lengths(case):
    """(cached lengths, new tokens) of a case's sequences, alike in every run of the case."""
    b, most = case["batch"], case["length"]
    r = random.Random(case["mix"])
    old = [most if not case["mix"] else r.randint(most // 3, most) for _ in range(b)]
    if case["mix"] and b > 2:
        old[1] = 0   # a sequence that has just come in
    new = [case["new"] if b == 1 else r.randint(max(1, case["new"] // 2), case["new"]) for _ in range(b)] \
        if case["op"] == "append" else None
    return old, new


def work(case):
    """Bytes and operations of one pass that no implementation can leave out."""
    if case["op"] == "rope":
        n = case["rows"] * case["heads"] * case["dim"]
        return {"bytes": 2 * n * (2 if case["dtype"] == "bf16" else 4) + 4 * case["rows"],
                "flops": 3 * case["rows"] * case["heads"] * case["rot"]}
    old, new = _lengths(case)
    if case["op"] == "append":
        n = 2 * sum(new) * case["kv"] * case["dim"]
        return {"bytes": n * (3 if case["fmt"] == "e4m3" else 4), "flops": 2 * n}
    d, b, n, hq, hkv = 128, case["batch"], case["nodes"], case["heads"], case["kv"]
    tree_bytes = 4 * b * n * hkv * d if case["tree"] else 0
    seen = min(n, 7) if case["tree"] else 0   # a node's path
    cache_bytes = 2 * sum(old) * hkv * d + sum(-(-x // GROUP) for x in old) * 2 * hkv
    return {"bytes": cache_bytes + tree_bytes + 4 * b * n * hq * d,
            "flops": 4 * d * hq * n * (sum(old) + b * seen)}


# ------------------------------------------------------------------------------------ frequencies
SCALING = dict(theta=500000.0, factor=8.0, low=1.0, high=4.0, fast=32.0, original=8192)


def _frequencies(rot, scaling):
    """Radians a position of the rotary pairs, in 64 bits."""
    p = SCALING
    theta = p["theta"] * p["factor"] ** (rot / (rot - 2)) if scaling == "base" else p["theta"]
    f = theta ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=DEV) / rot)
    if scaling == "linear":
        f = f / p["factor"]
    elif scaling == "bands":   # long wavelengths slowed down, short ones kept, a blend between
        turns = p["original"] * f / (2 * math.pi)
        keep = ((turns - p["low"]) / (p["high"] - p["low"])).clamp(0, 1)
        f = keep * f + (1 - keep) * f / p["factor"]
    elif scaling == "ramp":    # a blend by pair index between the pairs that turn `fast` and `low` times
        at = lambda turns: rot * math.log(p["original"] / (turns * 2 * math.pi)) / (2 * math.log(p["theta"]))
        lo, hi = max(math.floor(at(p["fast"])), 0), min(math.ceil(at(p["low"])), rot - 1)
        j = torch.arange(rot // 2, dtype=torch.float64, device=DEV)
        slowed = ((j - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        f = (1 - slowed) * f + slowed * f / p["factor"]
    return f


def _amplitude(scaling):
    return 0.1 * math.log(SCALING["factor"]) + 1.0 if scaling == "ramp" else 1.0


def _table(rot, scaling):
    import eagle_tree_speculative_spec_gb300 as e3
    p = SCALING
    kind = dict(none=e3.ROPE_NONE, linear=e3.ROPE_LINEAR, base=e3.ROPE_BASE, bands=e3.ROPE_BANDS, ramp=e3.ROPE_RAMP)
    table = torch.empty(rot // 2, dtype=torch.int64, device=DEV)
    e3.eagle3_rope_table(table, theta=p["theta"], scaling=kind[scaling], factor=p["factor"], low_turns=p["low"],
                         high_turns=p["fast"] if scaling == "ramp" else p["high"], original_positions=p["original"])
    return table


# ------------------------------------------------------------------------------------ inputs
def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _exponents(amax):
    """Biased exponent e of the least power of two 2^(e - 127) with amax <= 448 * 2^(e - 127), at least 1."""
    m, x = torch.frexp(amax)                       # 448 = 0.875 * 2^9
    e = x.to(torch.int32) - torch.where(m <= 0.875, 9, 8) + 127
    return torch.where(amax > 0, e, 1).clamp(1, 254).to(torch.uint8)


def _pow2(e):
    return (e.to(torch.int32) << 23).view(torch.float32)   # (the bits of fp32's powers of two)


def _filled_cache(g, pages, kv, page, dim, spread):
    """An e4m3 pool as earlier appends left it: codes [pages, kv, page, dim], scales [pages, kv, page / 64]."""
    x = _randn(g, pages, kv, page, dim) * spread
    grouped = x.view(pages, kv, page // GROUP, GROUP, dim)
    e = _exponents(grouped.abs().amax(dim=(3, 4)))
    codes = (grouped / _pow2(e)[..., None, None]).view(pages, kv, page, dim).to(F8)
    return codes, e


def _block_table(g, lengths, page, columns):
    """Pages of a pool in random order: ([batch, columns] int32, pages of the pool).  Columns past a
    sequence's last page name no page."""
    need = [-(-n // page) for n in lengths]
    pages = sum(need) + 2
    order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    table = torch.full((len(lengths), columns), -1, dtype=torch.int32, device=DEV)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, pages


def _trees(seed, batch, nodes):
    """Parent arrays of random trees, at most six deep."""
    r = random.Random(seed)
    out = []
    for _ in range(batch):
        par, depth = [-1], [0]
        for i in range(1, nodes):
            p = r.choice([j for j in range(i) if depth[j] < 6])
            par.append(p)
            depth.append(depth[p] + 1)
        out.append(par)
    return torch.tensor(out, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    i32, bf = torch.int32, torch.bfloat16
    s = dict(case)
    if case["op"] == "rope":
        dt = bf if case["dtype"] == "bf16" else torch.float32
        x = _randn(g, case["rows"], case["pitch"], case["dim"]).to(dt)
        s.update(x=x[:, :case["heads"]],
                 out=torch.empty(case["rows"], case["heads"], case["dim"], dtype=dt, device=DEV),
                 positions=torch.randint(0, case["far"], (case["rows"],), generator=g, device=DEV, dtype=i32))
        if own:
            s["table"] = _table(case["rot"], case["scaling"])
        return s
    old, new = _lengths(case)
    if case["op"] == "append":
        kv, dim, page, total = case["kv"], case["dim"], case["page"], sum(new)
        columns = max(-(-(a + n) // page) for a, n in zip(old, new))
        table, pages = _block_table(g, [a + n for a, n in zip(old, new)], page, columns)
        starts = [sum(new[:b]) for b in range(len(new))]
        rows = _randn(g, total, 2 * kv, dim)   # the key and value part of the fused projection
        rows *= torch.exp(0.7 * _randn(g, 1, 2 * kv, dim)) * torch.exp(0.3 * _randn(g, total, 1, 1))
        rows = rows.to(bf)
        s.update(k=rows[:, :kv], v=rows[:, kv:], block_table=table, total=total,
                 row_start=torch.tensor(starts, dtype=i32, device=DEV), n_new=torch.tensor(new, dtype=i32, device=DEV),
                 cache_len=torch.tensor(old, dtype=i32, device=DEV), max_new=max(new))
        if case["fmt"] == "e4m3":
            (s["k_cache"], s["k_scale"]), (s["v_cache"], s["v_scale"]) = (
                _filled_cache(g, pages, kv, page, dim, 1.5) for _ in range(2))
        else:
            s["k_cache"], s["v_cache"] = (_randn(g, pages * page, kv, dim).to(bf) for _ in range(2))
            s["k_scale"] = s["v_scale"] = None
        if own:
            s["table"] = _table(case["rot"], case["scaling"]) if case["rot"] else None
        return s
    b, n, hq, kv, page, d = case["batch"], case["nodes"], case["heads"], case["kv"], case["page"], 128
    columns = -(-max(1, case["length"]) // page)
    table, pages = _block_table(g, old, page, columns)
    channels = torch.exp(0.5 * _randn(g, d))
    (s["k_cache"], s["k_scale"]), (s["v_cache"], s["v_scale"]) = (
        _filled_cache(g, pages, kv, page, d, channels if i == 0 else 1.0) for i in range(2))
    s.update(q=(1.5 * _randn(g, b, n, hq, d) / channels).to(bf), block_table=table, longest=case["length"],
             prefix_len=torch.tensor(old, dtype=i32, device=DEV), out=torch.empty(b, n, hq, d, dtype=bf, device=DEV),
             lse=torch.empty(b, n, hq, device=DEV), tree_k=None, tree_v=None, parents=None)
    if case["tree"]:
        s.update(tree_k=(_randn(g, b, n, kv, d) * channels).to(bf), tree_v=_randn(g, b, n, kv, d).to(bf),
                 parents=_trees(seed, b, n))
    return s


# ------------------------------------------------------------------------------------ one pass
def run(s):
    if own:
        return _own(s)
    return {"rope": _plain_rope, "append": _plain_append, "attn": _plain_attn}[s["op"]](s)


def _own(s):
    import eagle_tree_speculative_spec_gb300 as e3
    layout = e3.ROPE_HALF if s.get("layout") == "half" else e3.ROPE_INTERLEAVED
    if s["op"] == "rope":
        e3.eagle3_rope(s["x"], s["positions"], s["table"], s["out"], layout=layout, inverse=s["inverse"],
                       amplitude=_amplitude(s["scaling"]))
        return s["out"]
    if s["op"] == "append":
        e3.eagle3_append_kv(s["k"], s["v"], s["cache_len"], s["n_new"], s["block_table"], s["k_cache"], s["v_cache"],
                            max_new=s["max_new"], block_size=s["page"], k_scale=s["k_scale"], v_scale=s["v_scale"],
                            row_start=s["row_start"], rope_table=s["table"], rope_layout=layout,
                            rope_amplitude=_amplitude(s["scaling"]) if s["rot"] else 1.0)
        return _caches(s)
    e3.eagle3_verify_attn_fp8(s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["block_table"],
                              s["prefix_len"], s["out"], max_prefix_len=s["longest"], tree_k=s["tree_k"],
                              tree_v=s["tree_v"], parents=s["parents"], lse=s["lse"])
    return s["out"], s["lse"]


def _caches(s):
    if s["fmt"] == "bf16":
        return s["k_cache"], s["v_cache"]
    return s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]


def _rotated(x, positions, rot, layout, scaling, inverse=False):
    """fp32 rows [T, heads, dim] with their first `rot` dims rotated."""
    angle = positions.to(torch.float64)[:, None] * _frequencies(rot, scaling)
    angle = torch.remainder(angle, 2 * math.pi)
    amp = _amplitude(scaling)
    cos, sin = (torch.cos(angle) * amp).float()[:, None], (torch.sin(angle) * amp).float()[:, None]
    if inverse:
        sin = -sin
    y = x.float().clone()
    r = y[..., :rot]
    a, b = (r[..., :rot // 2], r[..., rot // 2:]) if layout == "half" else (r[..., 0::2], r[..., 1::2])
    first, second = a * cos - b * sin, b * cos + a * sin
    a.copy_(first)
    b.copy_(second)
    return y


def _plain_rope(s):
    y = _rotated(s["x"], s["positions"], s["rot"], s["layout"], s["scaling"], s["inverse"])
    return y.to(s["x"].dtype)


def _places(s):
    """Sequence, position, page and offset of every new token."""
    seq = torch.repeat_interleave(torch.arange(s["batch"], device=DEV), s["n_new"], output_size=s["total"])
    at = torch.arange(s["total"], device=DEV) - s["row_start"][seq] + s["cache_len"][seq]
    return seq, at, s["block_table"][seq, at // s["page"]].long(), at % s["page"]


def _plain_append(s):
    seq, at, page, off = _places(s)
    k = _rotated(s["k"], at, s["rot"], s["layout"], s["scaling"]) if s["rot"] else s["k"].float()
    v = s["v"].float()
    if s["fmt"] == "bf16":
        s["k_cache"][page * s["page"] + off] = k.to(torch.bfloat16)
        s["v_cache"][page * s["page"] + off] = v.to(torch.bfloat16)
        return s["k_cache"], s["v_cache"]
    last = s["cache_len"].long()
    part = last % GROUP                                     # older tokens of a sequence's first group
    p0 = s["block_table"].gather(1, (last // s["page"])[:, None])[:, 0].long()
    g0 = last % s["page"] // GROUP
    older = (torch.arange(GROUP, device=DEV) < part[:, None])[:, None, :, None]
    for cache, scale, x in ((s["k_cache"], s["k_scale"], k), (s["v_cache"], s["v_scale"], v)):
        pages, kv, size, dim = cache.shape
        groups = size // GROUP
        amax = torch.zeros(pages * groups, kv, device=DEV)
        amax.scatter_reduce_(0, (page * groups + off // GROUP)[:, None].expand(-1, kv), x.abs().amax(2), "amax")
        touched = torch.zeros(pages * groups, dtype=torch.bool, device=DEV)
        touched[page * groups + off // GROUP] = True
        before = scale.permute(0, 2, 1).reshape(pages * groups, kv)
        kept = torch.zeros(pages * groups, dtype=torch.bool, device=DEV)
        kept[p0 * groups + g0] = part > 0
        fresh = _exponents(amax)
        after = torch.where(kept[:, None], torch.maximum(before, fresh), fresh)
        after = torch.where(touched[:, None], after, before)
        # the older tokens of a group whose scale has grown
        block = cache.view(torch.uint8).view(pages, kv, groups, GROUP, dim)
        codes = block[p0, :, g0]
        ratio = _pow2(before[p0 * groups + g0]) / _pow2(after[p0 * groups + g0])
        again = (codes.view(F8).float() * ratio[..., None, None]).to(F8).view(torch.uint8)
        block[p0, :, g0] = torch.where(older, again, codes)
        scale.copy_(after.view(pages, groups, kv).permute(0, 2, 1))
        q = (x / _pow2(after[page * groups + off // GROUP])[..., None]).to(F8)
        cache.view(torch.uint8)[page, :, off] = q.view(torch.uint8)
    return s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]


def _read(cache, scale, table, length):
    """The first `length` keys or values that the pages of `table` [..., columns] stand for: [..., kv, length, dim]."""
    pages, kv, size, dim = cache.shape
    ids = table.long().clamp_min(0)
    x = cache.view(torch.uint8)[ids].view(F8).float() * _pow2(scale[ids]).repeat_interleave(GROUP, -1)[..., None]
    x = x.transpose(-4, -3)                       # [..., kv, columns, size, dim]
    return x.flatten(-3, -2)[..., :length, :]


def _plain_attn(s):
    b, n, hq, d = s["q"].shape
    kv = s["kv"]
    q = s["q"].float().view(b, n, kv, hq // kv, d).permute(0, 2, 1, 3, 4).reshape(b, kv, n * (hq // kv), d)
    k = _read(s["k_cache"], s["k_scale"], s["block_table"], s["longest"])
    v = _read(s["v_cache"], s["v_scale"], s["block_table"], s["longest"])
    hidden = torch.arange(s["longest"], device=DEV) >= s["prefix_len"][:, None]
    v = v.masked_fill(hidden[:, None, :, None], 0.0)
    z = torch.matmul(q, k.transpose(2, 3)).masked_fill_(hidden[:, None, None, :], -math.inf)
    if s["tree"]:
        sees = torch.eye(n, dtype=torch.bool, device=DEV).repeat(b, 1, 1)
        for i in range(1, n):
            sees[:, i] |= sees[torch.arange(b, device=DEV), s["parents"][:, i].long()]
        zt = torch.matmul(q, s["tree_k"].float().permute(0, 2, 3, 1))
        zt = zt.view(b, kv, n, hq // kv, n).masked_fill(~sees[:, None, :, None, :], -math.inf)
        z = torch.cat([z, zt.view(b, kv, -1, n)], 3)
        v = torch.cat([v, s["tree_v"].float().transpose(1, 2)], 2)
    z = z * d ** -0.5
    high = z.amax(3, keepdim=True)
    high = torch.where(high > -math.inf, high, 0.0)
    p = torch.exp(z - high)
    total = p.sum(3, keepdim=True)
    out = torch.matmul(p, v) / torch.where(total > 0, total, 1.0)
    lse = (high + torch.log(total))[..., 0]
    out = out.view(b, kv, n, hq // kv, d).permute(0, 2, 1, 3, 4).reshape(b, n, hq, d)
    return out.to(torch.bfloat16), lse.view(b, kv, n, -1).transpose(1, 2).reshape(b, n, hq).contiguous()


# ------------------------------------------------------------------------------------ 64 bits
def _radians(case):
    """Each pair's angle a position, pair by pair."""
    p, rot, kind = SCALING, case["rot"], case["scaling"]
    bound = {t: rot * math.log(p["original"] / (2 * math.pi * p[t])) / (2 * math.log(p["theta"])) for t in ("fast", "low")}
    lo, hi = max(math.floor(bound["fast"]), 0), min(math.ceil(bound["low"]), rot - 1)
    out = []
    for j in range(rot // 2):
        base = p["theta"] if kind != "base" else p["theta"] * math.pow(p["factor"], rot / (rot - 2))
        w = math.exp(-2 * j / rot * math.log(base))
        slow = w / p["factor"]
        if kind == "linear":
            w = slow
        elif kind == "bands":
            wavelength = 2 * math.pi / w
            if wavelength > p["original"] / p["low"]:
                w = slow
            elif wavelength > p["original"] / p["high"]:
                mix = (p["original"] / wavelength - p["low"]) / (p["high"] - p["low"])
                w = (1 - mix) * slow + mix * w
        elif kind == "ramp":
            mix = min(max((j - lo) / max(hi - lo, 0.001), 0.0), 1.0)
            w = mix * slow + (1 - mix) * w
        out.append(w)
    return torch.tensor(out, dtype=torch.float64, device=DEV)


def _values(cache, scale, pages, length):
    """[kv, length, dim]: what the first `length` positions of a list of pages stand for, page by page."""
    kv, size, dim = cache.shape[1:]
    out = torch.zeros(kv, max(1, len(pages)) * size, dim, dtype=torch.float64, device=DEV)
    for i, p in enumerate(pages):
        for g in range(size // GROUP):
            at = slice(g * GROUP, (g + 1) * GROUP)
            factor = torch.exp2(scale[p, :, g].to(torch.float64) - 127)
            to = i * size + g * GROUP
            out[:, to:to + GROUP] = cache[p, :, at].to(torch.float64) * factor[:, None, None]
    return out[:, :length]


def _turned(x, positions, case, inverse=False):
    """Each pair as a complex number, multiplied by its position's."""
    rot, f64 = case["rot"], torch.float64
    y = x.to(f64).clone()
    if rot == 0:
        return y
    j = torch.arange(rot // 2, device=DEV)
    first, second = (j, j + rot // 2) if case["layout"] == "half" else (2 * j, 2 * j + 1)
    angle = positions.to(f64)[:, None] * _radians(case)
    w = torch.polar(torch.full_like(angle, _amplitude(case["scaling"])), -angle if inverse else angle)
    z = torch.complex(y[..., first], y[..., second]) * w[:, None]
    y[..., first], y[..., second] = z.real, z.imag
    return y


def exact(case, seed):
    """The operators' definitions, sequence by sequence and group by group, in 64 bits."""
    s = prepare(case, seed)
    f64 = torch.float64
    if case["op"] == "rope":
        return _turned(s["x"], s["positions"], case, case["inverse"])
    old, new = _lengths(case)
    if case["op"] == "append":
        page, kv = case["page"], case["kv"]
        table = s["block_table"].tolist()
        k_out, v_out = s["k_cache"].to(f64), s["v_cache"].to(f64)
        at = 0
        for b, (have, more) in enumerate(zip(old, new)):
            where = torch.arange(have, have + more, device=DEV)
            k = _turned(s["k"][at:at + more], where, case)
            v = s["v"][at:at + more].to(f64)
            at += more
            ids = torch.tensor(table[b], device=DEV)[where // page]
            if case["fmt"] == "bf16":
                k_out[ids * page + where % page] = k
                v_out[ids * page + where % page] = v
                continue
            for out, scale, x in ((k_out, s["k_scale"], k), (v_out, s["v_scale"], v)):
                # the first group, which may hold older tokens, then the whole groups behind it at once
                head = min(more, -have % GROUP)
                if head:
                    pid, g = table[b][have // page], have % page // GROUP
                    lo = have % GROUP
                    e_old = scale[pid, :, g].to(f64) - 127
                    e = torch.maximum(e_old, _least(x[:head].abs().amax((0, 2))))
                    rows = out[pid, :, g * GROUP:(g + 1) * GROUP]
                    rows[:, :lo] *= torch.exp2(e_old - e)[:, None, None]
                    rows[:, lo:lo + head] = x[:head].transpose(0, 1) / torch.exp2(e)[:, None, None]
                if more > head:
                    rest, pos = x[head:], where[head:]
                    full = torch.zeros(-(-(more - head) // GROUP) * GROUP, *rest.shape[1:], dtype=f64, device=DEV)
                    full[:more - head] = rest
                    e = _least(full.view(-1, GROUP, *rest.shape[1:]).abs().amax((1, 3)))
                    step = torch.exp2(e).repeat_interleave(GROUP, 0)[:more - head, :, None]
                    out[ids[head:], :, pos % page] = rest / step
        return (k_out, v_out) if case["fmt"] == "bf16" else (k_out, v_out, None, None)
    b, n, hq, d = s["q"].shape
    kv = case["kv"]
    rep = hq // kv
    out = torch.zeros(b, n, hq, d, dtype=f64, device=DEV)
    lse = torch.full((b, n, hq), -math.inf, dtype=f64, device=DEV)
    for i in range(b):
        pages = s["block_table"][i, :-(-old[i] // case["page"])].tolist()
        k = _values(s["k_cache"], s["k_scale"], pages, old[i])
        v = _values(s["v_cache"], s["v_scale"], pages, old[i])
        sees = torch.ones(n, old[i], dtype=torch.bool, device=DEV)
        if case["tree"]:
            k = torch.cat([k, s["tree_k"][i].to(f64).transpose(0, 1)], 1)
            v = torch.cat([v, s["tree_v"][i].to(f64).transpose(0, 1)], 1)
            par = s["parents"][i].tolist()
            own_path = torch.zeros(n, n, dtype=torch.bool)
            for node in range(n):
                at = node
                while at >= 0:
                    own_path[node, at] = True
                    at = par[at]
            sees = torch.cat([sees, own_path.to(DEV)], 1)
        if k.shape[1] == 0:
            continue
        for h in range(hq):
            z = (s["q"][i, :, h].to(f64) @ k[h // rep].t()) / math.sqrt(d)
            z = z.masked_fill(~sees, -math.inf)
            lse[i, :, h] = torch.logsumexp(z, 1)
            out[i, :, h] = torch.softmax(z, 1) @ v[h // rep]
    return out, lse


def _least(amax):
    """Least integer e with amax <= 448 * 2^e, at least -126."""
    e = torch.ceil(torch.log2(amax.clamp_min(1e-300) / 448)).clamp_min(-126)
    e = torch.where(amax > 448 * torch.exp2(e), e + 1, e)
    return torch.where((e > -126) & (amax <= 448 * torch.exp2(e - 1)), e - 1, e)
