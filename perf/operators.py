"""Measured cases of the mixture-of-experts and 8-bit projection operators.

The operators, as the feed-forward part of a mixture-of-experts target (or one with 8-bit
projections) runs them over the nodes of a batch of verified trees, or over single tokens:

  route     top-k experts of every row, their weights, and the rows sorted by expert
  grouped   matrix products grouped by expert over ragged row counts (SwiGLU gate + up with the
            rows gathered, or one product over rows already in expert order)
  combine   each row's weighted sum of its experts' outputs, plus the residual stream
  quantize  bf16 rows to e4m3 with one fp32 scale for each row and 128 columns
  fp8       e4m3 matrix product with a scale for each row and 128 columns of x and for each
            128 x 128 block of W, with the epilogues of the bf16 projections

``own`` selects between the plain forms (elementary torch operations in 32 bits) and the calls of
this package.  All sizes are rows x columns of the operation itself: 3840 rows are 64 trees of 60
nodes, 4096 and 14336 the hidden and feed-forward widths of the benchmark's target.
"""
import math

import torch

own = False

DEV = "cuda"
F8 = torch.float8_e4m3fn
F8_MAX = 448.0
BLOCK = 128


# ------------------------------------------------------------------------------------ cases
def listed():
    return [
        # one token of one sequence: the latency of a router call
        dict(name="route-1", op="route", rows=1, experts=64, top_k=8, scoring="softmax", renormalize=True, pad=0,
             masked=0),
        # 64 trees of 60 nodes in a padded batch, many experts, some of them switched off
        dict(name="route-3840", op="route", rows=3840, experts=256, top_k=8, scoring="sigmoid", renormalize=True,
             pad=131, masked=3),
        # one token: eight experts of one row each, gate + up
        dict(name="grouped-up-1", op="grouped", rows=1, experts=64, top_k=8, n=1024, k=4096, swiglu=True, skew=0.0),
        # one tree of 60 nodes: a few rows for every expert, down
        dict(name="grouped-down-60", op="grouped", rows=60, experts=64, top_k=8, n=4096, k=1024, swiglu=False,
             skew=0.5),
        # 64 trees of 60 nodes, gate + up: hundreds of rows for every expert
        dict(name="grouped-up-3840", op="grouped", rows=3840, experts=64, top_k=8, n=1024, k=4096, swiglu=True,
             skew=0.5),
        # ragged: odd sizes, experts of very unlike popularity, some without rows
        dict(name="grouped-down-1537", op="grouped", rows=1537, experts=40, top_k=3, n=2050, k=1400, swiglu=False,
             skew=2.0),
        # one tree of 60 nodes
        dict(name="combine-60", op="combine", rows=60, top_k=8, d=4096, residual=True, missing=0.0),
        # 64 trees of 60 nodes, a few experts missing
        dict(name="combine-3840", op="combine", rows=3840, top_k=8, d=4096, residual=True, missing=0.02),
        # single tokens of a batch of 64
        dict(name="quantize-64", op="quantize", rows=64, k=4096),
        # 64 trees of 60 nodes, the down projection's input
        dict(name="quantize-3840", op="quantize", rows=3840, k=14336),
        # single tokens of a batch of 8, the fused q/k/v projection
        dict(name="fp8-8", op="fp8", m=8, n=6144, k=4096, epilogue="bf16"),
        # 64 trees of 60 nodes, the gate + up projection
        dict(name="fp8-3840", op="fp8", m=3840, n=14336, k=4096, epilogue="swiglu"),
    ]


def _log(rng, lo, hi, step=1):
    """A multiple of `step` in [lo, hi], even over its logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(step, min(hi // step * step, round(v / step) * step))


def _cost(case):
    w = work(case)
    return w["bytes"] / 6.8e12 + w["flops"] / 1.7e15


def draw(rng):
    most = max(_cost(c) for c in listed() if c["op"] == "fp8")
    while True:
        op = rng.choice(["route", "grouped", "grouped", "combine", "quantize", "fp8", "fp8"])
        if op == "route":
            e = _log(rng, 4, 512)
            rows = _log(rng, 1, 3840)
            c = dict(op=op, rows=rows, experts=e, top_k=rng.randint(1, min(16, e)),
                     scoring=rng.choice(["softmax", "sigmoid"]), renormalize=rng.random() < 0.6,
                     pad=rng.choice([0, 0, rng.randint(0, rows)]), masked=rng.choice([0, rng.randint(0, e // 2)]))
        elif op == "grouped":
            e = _log(rng, 2, 128)
            c = dict(op=op, rows=_log(rng, 1, 3840), experts=e, top_k=rng.randint(1, min(8, e)),
                     n=_log(rng, 128, 4096), k=_log(rng, 128, 4096, 8), swiglu=rng.random() < 0.5,
                     skew=rng.choice([0.0, 0.5, 2.0]))
            if c["experts"] * c["n"] * c["k"] > 1 << 29:   # at most 1 GB of weights (2 GB with SwiGLU)
                continue
        elif op == "combine":
            c = dict(op=op, rows=_log(rng, 1, 3840), top_k=rng.randint(1, 16), d=_log(rng, 64, 8192),
                     residual=rng.random() < 0.6, missing=rng.choice([0.0, 0.1, 0.5]))
        elif op == "quantize":
            c = dict(op=op, rows=_log(rng, 1, 3840), k=_log(rng, 16, 14336, 16))
        else:
            c = dict(op=op, m=_log(rng, 1, 3840), n=_log(rng, 64, 14336), k=_log(rng, 128, 14336, 16),
                     epilogue=rng.choice(["bf16", "f32", "residual", "swiglu"]))
        if _cost(c) <= most:
            return c


def work(case):
    """Bytes and operations of one pass that no implementation can leave out."""
    op = case["op"]
    if op == "route":
        t, e, k = case["rows"], case["experts"], case["top_k"]
        return {"bytes": 4 * (t * e + 4 * t * k + e + 1), "flops": 4 * t * e}
    if op == "grouped":
        t, e, kk, n, k = case["rows"], case["experts"], case["top_k"], case["n"], case["k"]
        slots, mats = t * kk, 2 if case["swiglu"] else 1
        used = min(e, slots)   # experts with rows, at the most
        x_rows = t if case["swiglu"] else slots
        return {"bytes": 2 * (used * mats * n * k + x_rows * k + slots * n), "flops": 2 * slots * mats * n * k}
    if op == "combine":
        t, k, d = case["rows"], case["top_k"], case["d"]
        y = int(t * k * (1 - case["missing"]))
        return {"bytes": 2 * d * (y + t + (t if case["residual"] else 0)) + 8 * t * k, "flops": 2 * y * d}
    if op == "quantize":
        t, k = case["rows"], case["k"]
        return {"bytes": 3 * t * k + 4 * t * -(-k // BLOCK), "flops": 2 * t * k}
    m, n, k = case["m"], case["n"], case["k"]
    mats = 2 if case["epilogue"] == "swiglu" else 1
    out = 4 if case["epilogue"] == "f32" else 4 if case["epilogue"] == "residual" else 2   # residual: read + write
    kb = -(-k // BLOCK)
    return {"bytes": m * k + mats * n * k + out * m * n + 4 * kb * (m + mats * -(-n // BLOCK)),
            "flops": 2 * m * mats * n * k}


# ------------------------------------------------------------------------------------ inputs
def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _quantized(v, rows_per_scale):
    """(e4m3 values, scales [row blocks, k blocks]) of a [rows, k] fp32 tensor."""
    r, k = v.shape
    rb, kb = -(-r // rows_per_scale), -(-k // BLOCK)
    p = torch.zeros(rb * rows_per_scale, kb * BLOCK, device=DEV)
    p[:r, :k] = v
    p = p.view(rb, rows_per_scale, kb, BLOCK)
    s = p.abs().amax(dim=(1, 3)) / torch.full((), F8_MAX, device=DEV)
    s = torch.where(s > 0, s, torch.ones_like(s))
    q = (p / s[:, None, :, None]).clamp(-F8_MAX, F8_MAX)
    return q.view(rb * rows_per_scale, kb * BLOCK)[:r, :k].to(F8).contiguous(), s.contiguous()


def _assignment(g, rows, experts, top_k, skew):
    """Distinct experts of every row, popular ones more often with `skew`: (ids [rows, top_k])."""
    pop = skew * _randn(g, 1, experts)
    noise = torch.rand(rows, experts, generator=g, device=DEV).clamp_min(1e-20)
    return torch.topk(pop - torch.log(-torch.log(noise)), top_k, dim=1).indices


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    op = case["op"]
    i32, f32, bf = torch.int32, torch.float32, torch.bfloat16
    s = dict(case)
    if op == "route":
        t, e, k = case["rows"], case["experts"], case["top_k"]
        logits = 1.5 * _randn(g, t, e) + 0.5 * _randn(g, 1, e)
        if case["masked"]:   # experts that are switched off for every row
            off = torch.randperm(e, generator=g, device=DEV)[:case["masked"]]
            logits[:, off] = -math.inf
        s.update(logits=logits, num_rows=torch.full((1,), t - case["pad"], dtype=i32, device=DEV) if case["pad"] else None,
                 topk_ids=torch.empty(t, k, dtype=i32, device=DEV), topk_weights=torch.empty(t, k, dtype=f32, device=DEV),
                 offsets=torch.empty(e + 1, dtype=i32, device=DEV), sorted_rows=torch.empty(t * k, dtype=i32, device=DEV),
                 slots=torch.empty(t, k, dtype=i32, device=DEV))
    elif op == "grouped":
        t, e, kk, n, k = case["rows"], case["experts"], case["top_k"], case["n"], case["k"]
        flat = _assignment(g, t, e, kk, case["skew"]).reshape(-1)
        order = torch.argsort(flat, stable=True)
        counts = torch.bincount(flat, minlength=e)
        offsets = torch.zeros(e + 1, dtype=i32, device=DEV)
        offsets[1:] = torch.cumsum(counts, 0)
        w = [(_randn(g, e, n, k) * k ** -0.5).to(bf) for _ in range(2 if case["swiglu"] else 1)]
        x = _randn(g, t if case["swiglu"] else t * kk, k).to(bf)
        s.update(x=x, w=w[0], w2=w[1] if case["swiglu"] else None, offsets=offsets, largest=int(counts.max()),
                 row_ids=(order // kk).to(i32) if case["swiglu"] else None,
                 out=torch.empty(t * kk, n, dtype=bf, device=DEV))
    elif op == "combine":
        t, k, d = case["rows"], case["top_k"], case["d"]
        slots = torch.randperm(t * k, generator=g, device=DEV).view(t, k).to(i32)
        weights = torch.softmax(_randn(g, t, k), dim=1)
        gone = torch.rand(t, k, generator=g, device=DEV) < case["missing"]
        slots[gone] = -1
        weights[gone] = 0
        s.update(y=_randn(g, t * k, d).to(bf), slots=slots, weights=weights,
                 res=_randn(g, t, d).to(bf) if case["residual"] else None, out=torch.empty(t, d, dtype=bf, device=DEV))
    elif op == "quantize":
        t, k = case["rows"], case["k"]
        # activations: rows of unlike magnitude, a few columns far above the rest
        x = _randn(g, t, k) * torch.exp(_randn(g, t, 1))
        x = x * torch.where(torch.rand(1, k, generator=g, device=DEV) < 0.01, 20.0, 1.0)
        s.update(x=x.to(bf), q=torch.empty(t, k, dtype=F8, device=DEV),
                 scale=torch.empty(-(-k // BLOCK), t, dtype=f32, device=DEV))
    else:
        m, n, k = case["m"], case["n"], case["k"]
        epi = case["epilogue"]
        xq, xs = _quantized(_randn(g, m, k) * torch.exp(0.5 * _randn(g, m, 1)), 1)
        ws = [_quantized(_randn(g, n, k) * k ** -0.5, BLOCK) for _ in range(2 if epi == "swiglu" else 1)]
        s.update(x=xq, x_scale=xs.t().contiguous(), w=ws[0][0], w_scale=ws[0][1],
                 w2=ws[1][0] if epi == "swiglu" else None, w2_scale=ws[1][1] if epi == "swiglu" else None,
                 res=_randn(g, m, n).to(bf) if epi == "residual" else None,
                 out=torch.empty(m, n, dtype=f32 if epi == "f32" else bf, device=DEV))
    return s


# ------------------------------------------------------------------------------------ one pass
def run(s):
    op = s["op"]
    if own:
        return _own(s)
    if op == "route":
        return _plain_route(s)
    if op == "grouped":
        return _plain_grouped(s)
    if op == "combine":
        return _plain_combine(s)
    if op == "quantize":
        return _plain_quantize(s)
    return _plain_fp8(s)


def _own(s):
    import eagle_tree_speculative_spec_gb300 as e3
    op = s["op"]
    if op == "route":
        e3.eagle3_moe_route(s["logits"], s["topk_ids"], s["topk_weights"], s["offsets"], s["sorted_rows"], s["slots"],
                            scoring=e3.MOE_SOFTMAX if s["scoring"] == "softmax" else e3.MOE_SIGMOID,
                            renormalize=s["renormalize"], num_rows=s["num_rows"])
        return s["topk_ids"], s["topk_weights"], s["offsets"], s["sorted_rows"], s["slots"]
    if op == "grouped":
        e3.eagle3_grouped_linear(s["x"], s["w"], s["offsets"], s["out"],
                                 epilogue=e3.EPI_SWIGLU if s["swiglu"] else e3.EPI_BF16, w2=s["w2"],
                                 row_ids=s["row_ids"])
        return s["out"]
    if op == "combine":
        e3.eagle3_moe_combine(s["y"], s["slots"], s["weights"], s["out"], residual=s["res"])
        return s["out"]
    if op == "quantize":
        e3.eagle3_quantize_fp8(s["x"], s["q"], s["scale"])
        return s["q"], s["scale"]
    epi = {"bf16": e3.EPI_BF16, "f32": e3.EPI_F32, "residual": e3.EPI_BF16_RESIDUAL, "swiglu": e3.EPI_SWIGLU}
    e3.eagle3_linear_fp8(s["x"], s["x_scale"], s["w"], s["w_scale"], s["out"], epilogue=epi[s["epilogue"]], w2=s["w2"],
                         w2_scale=s["w2_scale"], residual=s["res"])
    return s["out"]


def _plain_route(s):
    z = s["logits"]
    t, e = z.shape
    k = s["top_k"]
    usable = torch.isfinite(z)
    if s["num_rows"] is not None:
        usable = usable & (torch.arange(t, device=DEV) < s["num_rows"])[:, None]
    z = torch.where(usable, z, -math.inf)
    top, ids = torch.sort(z, dim=1, descending=True, stable=True)   # equal logits: lowest expert first
    top, ids = top[:, :k], ids[:, :k]
    chosen = top > -math.inf
    if s["scoring"] == "softmax":
        high = torch.where(chosen[:, :1], top[:, :1], 0.0)
        score = torch.exp(top - high)
        total = torch.exp(z - high).sum(1, keepdim=True)
    else:
        score = torch.where(chosen, 1.0 / (1.0 + torch.exp(-top)), 0.0)
        total = torch.ones_like(top[:, :1])
    if s["renormalize"]:
        total = score.sum(1, keepdim=True)
    weights = torch.where(total > 0, score / total, 0.0)
    ids = torch.where(chosen, ids, -1).to(torch.int32)
    key = torch.where(chosen, ids, e).reshape(-1)
    order = torch.argsort(key, stable=True)
    offsets = torch.searchsorted(key[order], torch.arange(e + 1, device=DEV, dtype=key.dtype)).to(torch.int32)
    placed = torch.arange(t * k, device=DEV) < offsets[e]
    sorted_rows = torch.where(placed, order // k, -1).to(torch.int32)
    slots = torch.empty(t * k, dtype=torch.int32, device=DEV)
    slots[order] = torch.where(placed, torch.arange(t * k, device=DEV), -1).to(torch.int32)
    return ids, weights, offsets, sorted_rows, slots.view(t, k)


def _plain_grouped(s):
    """One batched product over the groups, each padded to the largest."""
    x, offsets = s["x"], s["offsets"]
    e, n, k = s["w"].shape
    m = s["out"].shape[0]
    slot = torch.arange(m, device=DEV, dtype=torch.int32)
    group = torch.searchsorted(offsets, slot, right=True) - 1
    at = slot - offsets[group]
    rows = torch.zeros(e, s["largest"], k, device=DEV)
    rows[group, at] = (x if s["row_ids"] is None else x[s["row_ids"]]).float()
    y = torch.bmm(rows, s["w"].float().transpose(1, 2))
    if s["w2"] is not None:
        y = y * torch.sigmoid(y) * torch.bmm(rows, s["w2"].float().transpose(1, 2))
    return y[group, at].to(torch.bfloat16)


def _plain_combine(s):
    present = s["slots"] >= 0
    y = s["y"][s["slots"].clamp_min(0)].float()
    out = torch.where(present[..., None], y * s["weights"][..., None], 0.0).sum(1)
    if s["res"] is not None:
        out = out + s["res"].float()
    return out.to(torch.bfloat16)


def _plain_quantize(s):
    x = s["x"]
    t, k = x.shape
    kb = -(-k // BLOCK)
    p = torch.zeros(t, kb * BLOCK, device=DEV)
    p[:, :k] = x
    p = p.view(t, kb, BLOCK)
    scale = p.abs().amax(dim=2) / torch.full((), F8_MAX, device=DEV)   # (by a Python number it would multiply)
    scale = torch.where(scale > 0, scale, 1.0)
    q = (p / scale[..., None]).clamp(-F8_MAX, F8_MAX)
    return q.view(t, kb * BLOCK)[:, :k].to(F8).contiguous(), scale.t().contiguous()


def _plain_fp8(s):
    k = s["x"].shape[1]
    n = s["w"].shape[0]
    x = s["x"].float() * s["x_scale"].repeat_interleave(BLOCK, 0)[:k].t()

    def product(w, scale):
        full = scale.repeat_interleave(BLOCK, 0)[:n].repeat_interleave(BLOCK, 1)[:, :k]
        return torch.matmul(x, (w.float() * full).t())

    y = product(s["w"], s["w_scale"])
    epi = s["epilogue"]
    if epi == "f32":
        return y
    if epi == "swiglu":
        y = y * torch.sigmoid(y) * product(s["w2"], s["w2_scale"])
    if epi == "residual":
        y = y + s["res"].float()
    return y.to(torch.bfloat16)


# ------------------------------------------------------------------------------------ 64 bits
def exact(case, seed):
    """The operators' definitions, expert by expert and block by block, in 64 bits."""
    s = prepare(case, seed)
    op = case["op"]
    f64 = torch.float64
    if op == "route":
        z = s["logits"].to(f64).clone()
        t, k = z.shape[0], case["top_k"]
        z[t - case["pad"]:] = -math.inf
        weights = torch.zeros(t, k, dtype=f64, device=DEV)
        left = z.clone()
        for j in range(k):
            best, at = left.max(1)
            weights[:, j] = best
            left[torch.arange(t, device=DEV), at] = -math.inf
        if case["scoring"] == "softmax":
            lse = torch.logsumexp(weights if case["renormalize"] else z, 1, keepdim=True)
            weights = torch.exp(weights - lse)
        else:
            weights = torch.sigmoid(weights)
            if case["renormalize"]:
                weights = weights / weights.sum(1, keepdim=True)
        return None, torch.nan_to_num(weights, nan=0.0), None, None, None
    if op == "grouped":
        ends = s["offsets"].tolist()
        out = torch.zeros(s["out"].shape, dtype=f64, device=DEV)
        for e, (a, b) in enumerate(zip(ends, ends[1:])):
            if a == b:
                continue
            x = (s["x"][a:b] if s["row_ids"] is None else s["x"][s["row_ids"][a:b].long()]).to(f64)
            y = x @ s["w"][e].to(f64).t()
            if s["w2"] is not None:
                y = y / (1 + torch.exp(-y)) * (x @ s["w2"][e].to(f64).t())
            out[a:b] = y
        return out
    if op == "combine":
        out = torch.zeros(s["out"].shape, dtype=f64, device=DEV) if s["res"] is None else s["res"].to(f64)
        for j in range(case["top_k"]):
            at = s["slots"][:, j].long()
            has = at >= 0
            out[has] += s["weights"][has, j].to(f64)[:, None] * s["y"][at[has]].to(f64)
        return out
    if op == "quantize":
        x = s["x"].to(f64)
        scale = torch.stack([c.abs().amax(1) for c in x.split(BLOCK, 1)]) / F8_MAX
        scale = torch.where(scale > 0, scale, 1.0)
        return x / scale.t().repeat_interleave(BLOCK, 1)[:, :case["k"]], scale
    x = s["x"].to(f64)

    def product(w, scale):
        y = torch.zeros(case["m"], case["n"], dtype=f64, device=DEV)
        for b, (xb, wb) in enumerate(zip(x.split(BLOCK, 1), w.split(BLOCK, 1))):
            y.addcmul_(xb @ wb.to(f64).t(),
                       s["x_scale"][b].to(f64)[:, None] * scale[:, b].to(f64).repeat_interleave(BLOCK)[:case["n"]])
        return y

    y = product(s["w"], s["w_scale"])
    if case["epilogue"] == "swiglu":
        y = y / (1 + torch.exp(-y)) * product(s["w2"], s["w2_scale"])
    if case["epilogue"] == "residual":
        y = y + s["res"].to(f64)
    return y
