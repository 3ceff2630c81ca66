"""GPU numerics of the mixture-of-experts operators against the fp64 oracle.

Tolerances, from the arithmetic (u = 2^-24, half an fp32 step; a bf16 output adds 2^-8 of its value):
  route    ids, offsets, rows and slots exact.  A weight is a quotient of sums of at most E positive
           exponentials: an argument z - m is off by u |z - m|, expf by 2 steps (4 u), a sum of E / 32
           terms in order and 5 shuffles by (E / 32 + 5) u, quotient and factor by 2 u, in numerator
           and denominator: u (2 (R + 4) + E / 32 + 9) relative, R the largest |z - m| (or |z|).
  grouped  the k products are exact, each of at most k additions is off by at most one fp32 step
           (2 u, the tensor cores cut) of a partial sum <= S = sum |x| |w|: 2 u k S.  SwiGLU carries
           it through silu (slope at most 1.1) times up, and its own exponential (2^-20 relative).
  combine  top_k products and additions and the residual's: u (2 top_k + 1) sum |terms|.
"""
import numpy as np
import pytest
import torch

import eagle_tree_speculative_spec_gb300 as e3
from oracle import moe
from tests._util import require_gpu

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF16 = 2.0 ** -8
TINY = 2.0 ** -133
bf, f32, i32 = torch.bfloat16, torch.float32, torch.int32


def _np(t):
    return t.double().cpu().numpy()


# ----------------------------------------------------------------------------- route
def _route(z, k, sigmoid=False, renorm=True, scale=1.0, num_rows=None, **kw):
    T, E = z.shape
    dev = z.device
    o = dict(ids=torch.full((T, k), -7, dtype=i32, device=dev), w=torch.full((T, k), -7.0, device=dev),
             off=torch.full((E + 1,), -7, dtype=i32, device=dev), rows=torch.full((T * k,), -7, dtype=i32, device=dev),
             slots=torch.full((T, k), -7, dtype=i32, device=dev))
    st = torch.zeros(1, dtype=i32, device=dev)
    nr = None if num_rows is None else torch.tensor([num_rows], dtype=i32, device=dev)
    e3.eagle3_moe_route(z, o["ids"], o["w"], o["off"], o["rows"], o["slots"],
                        scoring=e3.MOE_SIGMOID if sigmoid else e3.MOE_SOFTMAX, renormalize=renorm, scale=scale,
                        num_rows=nr, dev_status=st, **kw)
    torch.cuda.synchronize()
    return o, int(st)


def _check_route(z, k, status=0, **kw):
    o, st = _route(z, k, **kw)
    assert st == status
    kw = dict(kw)
    kw["renormalize"] = kw.pop("renorm", True)
    ids, w, off, rows, slots = moe.route(z.cpu().numpy(), k, **kw)
    for name, want in (("ids", ids), ("off", off), ("rows", rows), ("slots", slots)):
        np.testing.assert_array_equal(o[name].cpu().numpy(), want, err_msg=name)
    zz = z.double().cpu().numpy()
    fin = np.where(np.isfinite(zz), zz, np.nan)
    R = 0.0
    if np.isfinite(zz).any():
        R = np.nanmax(np.abs(fin)) if kw.get("sigmoid") else np.nanmax(fin) - np.nanmin(fin)
    tol = U * (2 * (R + 4) + z.shape[1] / 32 + 9)
    err = np.abs(_np(o["w"]) - w)
    assert (err <= tol * np.abs(w) + 1e-37).all(), (err.max(), tol)


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 64, 8), (5, 33, 16), (31, 8, 2), (32, 512, 8), (33, 512, 16),
                                   (60, 20, 3), (64, 64, 6), (65, 128, 8), (200, 512, 16), (256, 30, 5), (257, 64, 8),
                                   (1000, 256, 8), (3840, 100, 4), (6000, 7, 7)])
@pytest.mark.parametrize("sigmoid,renorm", [(False, True), (True, False)])
def test_route(T, E, k, sigmoid, renorm):
    dev = require_gpu()
    g = torch.Generator().manual_seed(T + E)
    _check_route((2 * torch.randn(T, E, generator=g)).to(dev), k, sigmoid=sigmoid, renorm=renorm, scale=2.5)


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("T", [20, 75, 300])
def test_route_unavailable_and_tied(sigmoid, renorm, T):
    """Ties (among them -0 and +0), rows with fewer than k finite logits, with none, the lowest value."""
    dev = require_gpu()
    g = torch.Generator().manual_seed(3)
    z = torch.randint(-2, 3, (T, 40), generator=g).float()
    z[0::2] = torch.where(z[0::2] == 0, -0.0, z[0::2])
    z[1, 3:] = -float("inf")
    z[2] = float("nan")
    z[3, ::2] = float("inf")
    z[4] = -float("inf")
    z[5] = torch.finfo(f32).min
    z[6] = 1.0
    z[7, 5] = 80.0
    _check_route(z.to(dev), 6, sigmoid=sigmoid, renorm=renorm)


@pytest.mark.parametrize("T,num_rows", [(20, 0), (20, 7), (20, 20), (200, 0), (200, 111), (300, 0), (300, 33), (300, 299), (5000, 4001)])
def test_route_num_rows(T, num_rows):
    dev = require_gpu()
    z = torch.randn(T, 48, generator=torch.Generator().manual_seed(4)).to(dev)
    _check_route(z, 4, num_rows=num_rows)


@pytest.mark.parametrize("num_rows", [-1, 41])
def test_route_num_rows_out_of_range(num_rows):
    dev = require_gpu()
    z = torch.randn(40, 16, generator=torch.Generator().manual_seed(5)).to(dev)
    _check_route(z, 4, num_rows=num_rows, status=4)


def test_route_no_rows_and_pitched_logits():
    dev = require_gpu()
    o, st = _route(torch.empty(0, 16, device=dev), 4)
    assert st == 0 and (o["off"] == 0).all()
    wide = torch.randn(50, 96, generator=torch.Generator().manual_seed(6)).to(dev)
    _check_route(wide[:, 10:50], 5)


def test_route_own_workspace():
    """Without a workspace: eager calls on two streams in turn, captured and replayed between them."""
    dev = require_gpu()
    z = [torch.randn(T, 48, generator=torch.Generator().manual_seed(T)).to(dev) for T in (300, 700)]
    want = [_route(x, 4)[0] for x in z]
    outs = [{k: torch.empty_like(v) for k, v in w.items()} for w in want]
    call = lambda i, **kw: e3.eagle3_moe_route(z[i], *(outs[i][k] for k in ("ids", "w", "off", "rows", "slots")), **kw)
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
        call(0)
        call(1)
    for _ in range(20):
        for o in outs:
            for v in o.values():
                v.fill_(-7)
        torch.cuda.synchronize()
        call(0, stream=side)
        junk = torch.full((1 << 14,), 3, dtype=i32, device=dev)   # the current stream's, beside the side stream's calls
        call(1, stream=side)
        graph.replay()
        torch.cuda.synchronize()
        assert (junk == 3).all()
        for o, w in zip(outs, want):
            for k in w:
                assert torch.equal(o[k], w[k]), k


def test_route_many_rows():
    """More rows than a block per 32: several chunks a block."""
    dev = require_gpu()
    T, E, k = 152 * 32 * 2 + 77, 64, 2
    z = torch.randn(T, E, generator=torch.Generator().manual_seed(7))
    o, st = _route(z.to(dev), k)
    assert st == 0
    top, ids = torch.sort(z, dim=1, descending=True, stable=True)
    ids = ids[:, :k]
    order = torch.argsort(ids.reshape(-1), stable=True)
    assert torch.equal(o["ids"].cpu().long(), ids)
    assert torch.equal(o["rows"].cpu().long(), order // k)
    slots = torch.empty(T * k, dtype=torch.long)
    slots[order] = torch.arange(T * k)
    assert torch.equal(o["slots"].cpu().long().view(-1), slots)
    assert torch.equal(o["off"].cpu().long()[1:], torch.bincount(ids.reshape(-1), minlength=E).cumsum(0))


# ----------------------------------------------------------------------------- grouped products
def _offsets(counts, dev):
    return torch.tensor([0] + list(np.cumsum(counts)), dtype=i32, device=dev)


def _grouped(counts, n, k, swiglu, gather, seed=0, spare=0, pitch=0, n_src=None):
    dev = require_gpu()
    g = torch.Generator().manual_seed(seed)
    E, used = len(counts), int(sum(counts))
    m = used + spare
    n_src = n_src or max(1, m // 2)
    x = torch.randn(n_src if gather else m, k + pitch, generator=g).to(bf)
    w = (torch.randn(E, n, k, generator=g) * k ** -0.5).to(bf)
    w2 = (torch.randn(E, n, k, generator=g) * k ** -0.5).to(bf) if swiglu else None
    ids = torch.randint(0, n_src, (m,), generator=g, dtype=i32) if gather else None
    if gather:
        ids[used:] = -1
    off = _offsets(counts, dev)
    out = torch.full((m, n + pitch), 7.0, dtype=bf, device=dev)
    st = torch.zeros(1, dtype=i32, device=dev)
    xd = x.to(dev)
    e3.eagle3_grouped_linear(xd[:, :k], w.to(dev), off, out[:, :n], epilogue=e3.EPI_SWIGLU if swiglu else e3.EPI_BF16,
                             w2=None if w2 is None else w2.to(dev), row_ids=None if ids is None else ids.to(dev),
                             dev_status=st)
    torch.cuda.synchronize()
    assert int(st) == 0
    got = _np(out)
    assert (got[used:] == 7).all() and (got[:, n:] == 7).all(), "wrote outside the groups' rows"
    want, S, gate, up = moe.grouped_linear(_np(x[:, :k]), _np(w), off.cpu().numpy(), None if ids is None else ids.numpy(),
                                           None if w2 is None else _np(w2))
    tol = 2 * U * k * S
    if swiglu:
        tol = 1.1 * tol * (np.abs(up) + tol) + np.abs(moe.silu(gate)) * tol + 2.0 ** -20 * np.abs(want)
    tol = tol + BF16 * (np.abs(want) + tol) + TINY
    err = np.abs(got[:used, :n] - want)
    assert (err <= tol).all(), (float((err / tol).max()), float(err.max()))


@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("counts,n,k", [
    ([1], 128, 64),
    ([0, 1, 0], 8, 8),
    ([5, 0, 17, 1], 200, 72),
    ([16, 32, 15, 33], 256, 256),
    ([255, 256, 257, 0, 300], 130, 136),
    ([0, 0, 0], 64, 64),
    ([700, 2], 63, 520),
    ([2400, 1], 65, 64),               # ten row tiles of a group
])
def test_grouped(counts, n, k, swiglu, gather):
    _grouped(counts, n, k, swiglu, gather, seed=sum(counts) + n)


@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("counts,n,k", [
    ([1], 128, 1024), ([0, 1, 0, 2], 200, 2056), ([3, 17], 77, 1000), ([256], 64, 4096), ([250, 0, 40], 130, 1544),
    ([0, 0], 64, 2048), ([9, 8, 7, 6, 5], 500, 640), ([600], 40, 3000)])
def test_grouped_k_ranges(counts, n, k, swiglu, gather):
    """Few units and a long k: the k-blocks are cut over a cluster."""
    _grouped(counts, n, k, swiglu, gather, seed=n + k, spare=3, pitch=8 if gather else 0)


def test_grouped_spare_rows_and_pitches():
    _grouped([3, 40, 0, 9], 96, 128, False, True, spare=21, pitch=8)
    _grouped([3, 40, 0, 9], 96, 128, True, False, spare=21, pitch=8)


def test_grouped_odd_columns():
    """Odd output widths (no column pairs), odd and even pitches."""
    _grouped([20, 3], 77, 64, False, True)
    _grouped([20, 3], 77, 64, True, True, pitch=8)
    _grouped([1, 1], 1, 64, True, False)


def test_grouped_many_groups_and_waves():
    r = np.random.default_rng(8)
    counts = r.integers(0, 4, 512)
    _grouped(list(counts), 64, 64, False, True, n_src=37)
    _grouped(list(counts), 130, 64, True, True, n_src=37)
    _grouped(list(r.integers(0, 90, 30)), 700, 320, True, True)


def test_grouped_same_row_everywhere():
    _grouped([64, 64], 128, 128, False, True, n_src=1)


@pytest.mark.parametrize("offsets", [[1, 2, 3, 4], [0, 3, 2, 4], [0, 2, 3, 99], [0, -1, 3, 4]])
def test_grouped_bad_offsets(offsets):
    """Offsets that do not start at 0, decrease or pass m: flagged, nothing written."""
    dev = require_gpu()
    out = torch.full((4, 64), 7.0, dtype=bf, device=dev)
    st = torch.zeros(1, dtype=i32, device=dev)
    e3.eagle3_grouped_linear(torch.ones(4, 64, dtype=bf, device=dev), torch.ones(3, 64, 64, dtype=bf, device=dev),
                             torch.tensor(offsets, dtype=i32, device=dev), out, dev_status=st)
    torch.cuda.synchronize()
    assert int(st) == 0x20 and (out == 7).all()


def test_grouped_bad_row_id_voids_its_row_only():
    dev = require_gpu()
    g = torch.Generator().manual_seed(9)
    x, w = torch.randn(5, 64, generator=g).to(bf).to(dev), torch.randn(2, 64, 64, generator=g).to(bf).to(dev)
    off, good = torch.tensor([0, 3, 6], dtype=i32, device=dev), torch.tensor([0, 1, 2, 3, 4, 0], dtype=i32, device=dev)
    bad = good.clone()
    bad[1], bad[4] = 5, -1
    outs = []
    for ids in (good, bad):
        out, st = torch.zeros(6, 64, dtype=bf, device=dev), torch.zeros(1, dtype=i32, device=dev)
        e3.eagle3_grouped_linear(x, w, off, out, row_ids=ids, dev_status=st)
        torch.cuda.synchronize()
        outs.append((out, int(st)))
    assert outs[0][1] == 0 and outs[1][1] == 0x20
    keep = [0, 2, 3, 5]
    assert torch.equal(outs[0][0][keep], outs[1][0][keep])


def test_grouped_nan_stays_in_its_row():
    dev = require_gpu()
    x = torch.ones(40, 64, dtype=bf, device=dev)
    x[7, 3] = float("nan")
    x[9, 0] = float("inf")
    out = torch.zeros(40, 64, dtype=bf, device=dev)
    e3.eagle3_grouped_linear(x, torch.ones(2, 64, 64, dtype=bf, device=dev), _offsets([18, 22], dev), out)
    assert torch.isnan(out[7]).all() and torch.isinf(out[9]).all()
    rest = [i for i in range(40) if i not in (7, 9)]
    assert (out[rest] == 64).all()


# ----------------------------------------------------------------------------- combine
@pytest.mark.parametrize("T,k,d,residual,pitch", [
    (1, 1, 8, False, 0), (1, 8, 4096, True, 0), (60, 8, 4096, True, 0), (33, 16, 1032, False, 0), (7, 3, 2050, True, 0),
    (9, 5, 77, True, 0), (5, 2, 64, True, 8), (5, 2, 64, True, 2), (5, 2, 63, False, 1), (2, 9, 9000, True, 0)])
def test_combine(T, k, d, residual, pitch):
    dev = require_gpu()
    g = torch.Generator().manual_seed(T + k + d)
    n_slots = T * k + 3
    y = torch.randn(n_slots, d + pitch, generator=g).to(bf)[:, :d]
    slots = torch.randint(-1, n_slots, (T, k), generator=g, dtype=i32)   # the same slot may come twice
    slots[0, 0] = -1
    w = torch.randn(T, k, generator=g)
    res = torch.randn(T, d + pitch, generator=g).to(bf)[:, :d] if residual else None
    out = torch.full((T, d + pitch), 7.0, dtype=bf, device=dev)
    st = torch.zeros(1, dtype=i32, device=dev)
    dd = lambda t: None if t is None else torch.empty(t.shape[0], d + pitch, dtype=bf, device=dev)[:, :d].copy_(t)
    e3.eagle3_moe_combine(dd(y), slots.to(dev), w.to(dev), out[:, :d], residual=dd(res), dev_status=st)
    torch.cuda.synchronize()
    assert int(st) == 0 and (out[:, d:] == 7).all()
    want, S = moe.combine(_np(y), slots.numpy(), w.double().numpy(), None if res is None else _np(res))
    tol = U * (2 * k + 1) * S
    tol = tol + BF16 * (np.abs(want) + tol) + TINY
    assert (np.abs(_np(out[:, :d]) - want) <= tol).all()


def test_combine_empty_places_and_bad_slots():
    """An empty place adds nothing whatever its weight; a slot past the end is empty and flagged; out
    may be the residual."""
    dev = require_gpu()
    y = torch.full((2, 64), float("inf"), dtype=bf, device=dev)
    buf = torch.randn(3, 64, device=dev).to(bf)
    keep = buf.clone()
    slots = torch.tensor([[-1, -1], [-5, -1], [2, -1]], dtype=i32, device=dev)
    w = torch.full((3, 2), float("nan"), device=dev)
    st = torch.zeros(1, dtype=i32, device=dev)
    e3.eagle3_moe_combine(y, slots, w, buf, residual=buf, dev_status=st)
    torch.cuda.synchronize()
    assert int(st) == 0x20 and torch.equal(buf, keep)
    out = torch.full((3, 64), 7.0, dtype=bf, device=dev)
    e3.eagle3_moe_combine(y[:0], slots[:2].clone(), w[:2].clone(), out[:2])
    torch.cuda.synchronize()
    assert (out[:2] == 0).all() and (out[2] == 7).all()


# ----------------------------------------------------------------------------- together
def _layer(dev, T, d, F, E, k, seed=0):
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g)
    return dict(x=rnd(T, d).to(bf).to(dev), res=rnd(T, d).to(bf).to(dev), wr=(rnd(E, d) * d ** -0.5).to(bf).to(dev),
                wg=(rnd(E, F, d) * d ** -0.5).to(bf).to(dev), wu=(rnd(E, F, d) * d ** -0.5).to(bf).to(dev),
                wd=(rnd(E, d, F) * F ** -0.5).to(bf).to(dev), z=torch.empty(T, E, device=dev),
                ids=torch.empty(T, k, dtype=i32, device=dev), w=torch.empty(T, k, device=dev),
                off=torch.empty(E + 1, dtype=i32, device=dev), rows=torch.empty(T * k, dtype=i32, device=dev),
                slots=torch.empty(T, k, dtype=i32, device=dev), h=torch.zeros(T * k, F, dtype=bf, device=dev),
                y=torch.zeros(T * k, d, dtype=bf, device=dev), out=torch.empty(T, d, dtype=bf, device=dev),
                ws=torch.empty(1 << 20, dtype=torch.uint8, device=dev), ws_lin=torch.empty(64 << 20, dtype=torch.uint8, device=dev),
                n=torch.full((1,), T, dtype=i32, device=dev), st=torch.zeros(1, dtype=i32, device=dev))


def _run_layer(L):
    e3.eagle3_linear(L["x"], L["wr"], L["z"], epilogue=e3.EPI_F32, workspace=L["ws_lin"], dev_status=L["st"])
    e3.eagle3_moe_route(L["z"], L["ids"], L["w"], L["off"], L["rows"], L["slots"], num_rows=L["n"], workspace=L["ws"],
                        dev_status=L["st"])
    e3.eagle3_grouped_linear(L["x"], L["wg"], L["off"], L["h"], epilogue=e3.EPI_SWIGLU, w2=L["wu"], row_ids=L["rows"],
                             dev_status=L["st"])
    e3.eagle3_grouped_linear(L["h"], L["wd"], L["off"], L["y"], dev_status=L["st"])
    e3.eagle3_moe_combine(L["y"], L["slots"], L["w"], L["out"], residual=L["res"], dev_status=L["st"])


def _layer_ref(L, limit):
    ids, w, off, rows, slots = moe.route(L["z"].cpu().numpy(), L["ids"].shape[1], num_rows=limit)
    h = moe.grouped_linear(_np(L["x"]), _np(L["wg"]), off, rows, _np(L["wu"]))[0]
    y = moe.grouped_linear(h, _np(L["wd"]), off)[0]
    return moe.combine(y, slots, w, _np(L["res"]))[0]


def test_layer_eager_graph_and_side_stream():
    """Router, products and combination as a layer uses them: eagerly, captured into two graphs that
    share the buffers and replayed in turn with other inputs and row counts, and on a side stream."""
    dev = require_gpu()
    T, d, F, E, k = 70, 256, 192, 12, 3
    L = _layer(dev, T, d, F, E, k)

    def check(limit):
        torch.cuda.synchronize()
        assert int(L["st"]) == 0
        want = _layer_ref(L, limit)
        # two bf16 roundings of intermediates (h, y) and one of the output; values of order 1, sums over
        # F of rounded h: 2^-8 of S <= |y| sqrt(F)-like terms: 8 steps cover them
        err = np.abs(_np(L["out"]) - want)
        assert (err <= 8 * BF16 * (1 + np.abs(want))).all(), err.max()

    _run_layer(L)
    check(T)
    side = torch.cuda.Stream()
    graphs = []
    with torch.cuda.stream(side):
        for _ in range(2):
            gr = torch.cuda.CUDAGraph()
            with torch.cuda.graph(gr, stream=side):
                _run_layer(L)
            graphs.append(gr)
    for i, limit in enumerate((T, 40, 0, 65)):
        L["x"].copy_(torch.randn(T, d, generator=torch.Generator().manual_seed(50 + i)).to(bf))
        L["n"].fill_(limit)
        torch.cuda.synchronize()
        graphs[i % 2].replay()
        check(limit)
    L["n"].fill_(T)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        L["out"].zero_()
        _run_layer(L)
    check(T)
    first = L["out"].clone()
    for _ in range(3):   # bit-identical run to run
        _run_layer(L)
        torch.cuda.synchronize()
        assert torch.equal(first, L["out"])


def test_calls_on_two_streams_at_once():
    dev = require_gpu()
    layers = [_layer(dev, T, 256, 256, 16, 4, seed=T) for T in (300, 90)]
    for L in layers:
        _run_layer(L)
    torch.cuda.synchronize()
    want = [L["out"].clone() for L in layers]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for L, s in zip(layers, streams):
            L["out"].zero_()
        torch.cuda.synchronize()
        for L, s in zip(layers, streams):
            with torch.cuda.stream(s):
                _run_layer(L)
        torch.cuda.synchronize()
        for L, w in zip(layers, want):
            assert int(L["st"]) == 0 and torch.equal(L["out"], w)


# ----------------------------------------------------------------------------- borders
def _silu_tol(a, up):
    """silu(a) * up: the exponential is 2 + 1.2 |a| fp32 steps (2 u) off, division and product 3 more, the
    result is rounded to bf16; below -87.3 it is 0, an error of less than 2^-119 times up."""
    want = moe.silu(a) * up
    tol = (BF16 + 2 * U * (8 + 1.2 * np.abs(np.clip(a, -100, 100)))) * np.abs(want)
    return want, tol + np.where(a < -87, 2.0 ** -119, 0) * np.abs(up) + TINY


@pytest.mark.parametrize("n", [64, 256])   # single CTAs and pairs
def test_grouped_extreme_gates(n):
    """Gates from the lowest number to infinity: x[s] = (gate, up, 0, ...) and unit weights."""
    dev = require_gpu()
    gates = [0.0, -0.0, 1.0, -1.0, -20.0, -60.0, -80.0, -87.0, -87.5, -88.0, -89.0, -100.0, 88.0, 100.0, -1e30, -3e38]
    ups = [1.0, -2.0, 1e30, 0.0]
    pairs = [(a, u) for a in gates for u in ups] + [(3e38, 1.0), (3e38, 0.5)]
    x = torch.zeros(len(pairs), 64, dtype=bf)
    x[:, :2] = torch.tensor(pairs).to(bf)
    wg, wu = torch.zeros(1, n, 64, dtype=bf), torch.zeros(1, n, 64, dtype=bf)
    wg[:, :, 0] = 1
    wu[:, :, 1] = 1
    out = torch.empty(len(pairs), n, dtype=bf, device=dev)
    off = _offsets([len(pairs)], dev)
    e3.eagle3_grouped_linear(x.to(dev), wg.to(dev), off, out, epilogue=e3.EPI_SWIGLU, w2=wu.to(dev))
    want, tol = _silu_tol(_np(x[:, 0]), _np(x[:, 1]))
    assert (np.abs(_np(out) - want[:, None]) <= tol[:, None]).all()
    wg[:, :, 0] = 2   # the sum passes fp32's range: +inf
    e3.eagle3_grouped_linear(x.to(dev), wg.to(dev), off, out, epilogue=e3.EPI_SWIGLU, w2=wu.to(dev))
    assert (out[-2:] == float("inf")).all()


def test_offsets_past_32_bits():
    """Rows, weights and slots further than 2^31 elements from their first."""
    dev = require_gpu()
    g = torch.Generator().manual_seed(11)
    k, n, far = 4096, 1100, 600000
    x = torch.empty(far, k, dtype=bf, device=dev)
    ids = torch.tensor([far - 1, 0, far - 3], dtype=i32, device=dev)
    x[ids.long()] = torch.randn(3, k, generator=g).to(bf).to(dev)
    w = torch.empty(512, n, k, dtype=bf, device=dev)
    used = [0, 511]
    w[used] = (torch.randn(2, n, k, generator=g) * k ** -0.5).to(bf).to(dev)
    off = torch.ones(513, dtype=i32, device=dev)   # row 0 by group 0, rows 1 and 2 by group 511
    off[0], off[512] = 0, 3
    out = torch.empty(3, n, dtype=bf, device=dev)
    e3.eagle3_grouped_linear(x, w, off, out, row_ids=ids)
    want, S, _, _ = moe.grouped_linear(_np(x[ids.long()]), _np(w[used]), np.array([0, 1, 3]))
    tol = 2 * U * k * S
    assert (np.abs(_np(out) - want) <= tol + BF16 * (np.abs(want) + tol) + TINY).all()
    slots = torch.tensor([[far - 1, 0], [-1, far - 3]], dtype=i32, device=dev)
    res = torch.empty(2, k, dtype=bf, device=dev)
    e3.eagle3_moe_combine(x, slots, torch.ones(2, 2, device=dev), res)
    want = _np(x[ids.long()])
    want = np.stack([want[0] + want[1], want[2]])
    assert (np.abs(_np(res) - want) <= (BF16 + 4 * U) * (np.abs(want) + 1)).all()


def test_readme_example():
    """The documentation's mixture-of-experts and 8-bit example, run as written."""
    dev = require_gpu()
    import os
    import re

    from oracle import fp8
    from tests._util import ROOT
    text = open(os.path.join(ROOT, "README.md")).read()
    code = [b for b in re.findall(r"```python\n(.*?)```", text, flags=re.S) if "eagle3_moe_route" in b]
    assert len(code) == 1
    v = {}
    exec(code[0], v)
    torch.cuda.synchronize()
    L = dict(z=v["logits"], ids=v["ids"], x=v["x"], wg=v["wg"], wu=v["wu"], wd=v["wd"], res=v["res"])
    want = _layer_ref(L, v["T"])
    # as in the layer test above: two roundings of intermediates and one of the output
    assert (np.abs(_np(v["out"]) - want) <= 8 * BF16 * (1 + np.abs(want))).all()
    codes, scale = fp8.quantize(v["out"].float().cpu().numpy())
    y, S = fp8.linear(codes, scale, v["w8"].view(torch.uint8).cpu().numpy(), v["w_scale"].cpu().numpy())
    tol = (256 + 3 + scale.shape[0]) * U * S
    assert (np.abs(_np(v["proj"]) - y) <= tol + BF16 * (np.abs(y) + tol) + TINY).all()


# ----------------------------------------------------------------------------- as few k-blocks as ranks
def _leave_in_tmem(value):
    """Accumulators full of `value` in the tensor memory of every SM."""
    dev = require_gpu()
    x = torch.full((1024, 64), value, dtype=bf, device=dev)
    e3.eagle3_grouped_linear(x, torch.ones(1, 128 * 160, 64, dtype=bf, device=dev), _offsets([1024], dev),
                             torch.empty(1024, 128 * 160, dtype=bf, device=dev))


@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("k", [320, 328, 384, 392, 448, 456, 512, 576])
@pytest.mark.parametrize("counts,n", [([1], 64), ([1], 128), ([0, 1, 0], 200), ([2, 2], 1024), ([15], 128), ([16], 64),
                                      ([3, 28], 128)])
def test_grouped_short_k_ranges(counts, n, k, swiglu, gather):
    """5 to 9 k-blocks, where a cut over a cluster begins to pay: every rank has a block of its own, so that nothing
    of what an earlier call left in tensor memory (NaN, large sums) gets into the sums, and every run gives the
    same bits."""
    _leave_in_tmem(float("nan"))
    _grouped(counts, n, k, swiglu, gather, seed=n + k, spare=2)
    dev = require_gpu()
    g = torch.Generator().manual_seed(k)
    m = sum(counts)
    x, w, w2 = (torch.randn(*s, generator=g).to(bf).to(dev) for s in ((m, k), (len(counts), n, k), (len(counts), n, k)))
    ids = torch.arange(m, dtype=i32, device=dev) if gather else None
    outs = []
    for value in (1.0, 3e4, float("nan")):
        _leave_in_tmem(value)
        out = torch.empty(m, n, dtype=bf, device=dev)
        e3.eagle3_grouped_linear(x, w, _offsets(counts, dev), out, epilogue=e3.EPI_SWIGLU if swiglu else e3.EPI_BF16,
                                 w2=w2 if swiglu else None, row_ids=ids)
        outs.append(out)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


@pytest.mark.parametrize("T", [33, 61, 97, 130, 191, 225, 256])
@pytest.mark.parametrize("k", [1, 3, 7])
def test_route_cluster_with_uneven_ends(T, k):
    """One launch of a cluster whose last rows, empty places and filler end in the middle of a warp, ten times over."""
    dev = require_gpu()
    z = torch.randn(T, 24, generator=torch.Generator().manual_seed(T + k))
    z[::3, k // 2:] = -float("inf")   # every third row has too few
    z = z.to(dev)
    _check_route(z, k, num_rows=T - 5)
    want = _route(z, k, num_rows=T - 5)[0]
    for _ in range(10):
        got = _route(z, k, num_rows=T - 5)[0]
        assert all(torch.equal(got[n], want[n]) for n in want)


@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("n,k", [(128, 64), (640, 64), (64, 4096)])   # single CTAs, pairs, k over a cluster
@pytest.mark.parametrize("offsets", [[0, 2 ** 31 - 1, -2 ** 31, 4], [-2 ** 31, 2 ** 31 - 1, 0, 4], [0, 2, 2 ** 31 - 1, 4],
                                     [2 ** 31 - 1, -2 ** 31, 2 ** 31 - 1, -2 ** 31], [0, 4, 4, -1]])
def test_grouped_wild_offsets(offsets, n, k, gather, swiglu):
    """Offsets whose differences pass 32 bits: flagged, nothing written, and the next call is in order."""
    dev = require_gpu()
    x, w = torch.ones(4, k, dtype=bf, device=dev), torch.ones(3, n, k, dtype=bf, device=dev)
    out, st = torch.full((4, n), 7.0, dtype=bf, device=dev), torch.zeros(1, dtype=i32, device=dev)
    ids = torch.arange(4, dtype=i32, device=dev) if gather else None
    call = lambda off: e3.eagle3_grouped_linear(x, w, torch.tensor(off, dtype=i32, device=dev), out, row_ids=ids,
                                                epilogue=e3.EPI_SWIGLU if swiglu else e3.EPI_BF16,
                                                w2=w if swiglu else None, dev_status=st)
    call(offsets)
    torch.cuda.synchronize()
    assert int(st) == 0x20 and (out == 7).all()
    st.zero_()
    call([0, 1, 1, 4])
    torch.cuda.synchronize()
    assert int(st) == 0 and (out == (k * k if swiglu else k)).all()
