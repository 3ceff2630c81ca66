"""GPU numerics of the 8-bit paged cache's operators against the fp64 oracle.

Tolerances, from the arithmetic (u = 2^-24, half an fp32 step relative to a value):
Rotations.  The angle is exact to 2^-33 turns; from the nearest quarter turn (at most pi / 4) it is rounded twice in
fp32, off by at most (1/2 + 1) pi / 4 u + 2^-32 pi; the series leave out less than 2^-25 and round once at the end, to half a
step: sine and cosine within 1.2 + 0.1 + 0.5 + 0.5 u, times the amplitude one rounding: together
below ANGLE = 7 u for each of the two terms, and 3 roundings of the products and the sum: an element is off by at most
amplitude (|a| + |b|) 10 u, and half a step of the type it is stored in (2^-8 of a bf16 value, 2^-4 of an e4m3 one or 2^-10 of its
scale's unit).  Positions beyond 2^20 add the table's own 2^-53 of a turn each.
Attention.  A score: its products are exact, but for queries (and tree keys) in two 8-bit parts: the row is scaled so
that its largest magnitude is above 224, and what is below 2^-2 there is rounded to steps of 2^-9, so off by at most 2^-10,
2^-17 of the row's largest (of the tree's largest key element); 128 additions, each off
by at most one step (2 u) of the sum of magnitudes S, and 6 roundings of scales and the maximum's subtraction: (256 + 6) u S
in natural units, and the 2^x unit is within 2^-22: a weight is off by w = (262 u S + 2^-17 (Qmax |k|_1 + Kmax |q|_1) scale + 2^-21) of
itself, and by 2^-11 where it is rounded to fp16 for V (2^-31 of the largest weight below fp16's normal range, n 2^-31 in all).
With M the weighted mean magnitude of V, an output is off by (2 w + 2^-11 + (n + 64) 2 u) M + n 2^-31 max|V| before
bf16's half step; the logarithm by w + (n + 64) 2 u + 8 u |lse|.
"""
import math

import numpy as np
import pytest
import torch

import eagle_tree_speculative_spec_gb300 as e3
from eagle_tree_speculative_spec_gb300 import _lib
from oracle import fp8, kv
from tests._util import require_gpu

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF16 = 2.0 ** -8
bf, f32, i32, i64, u8, f8 = torch.bfloat16, torch.float32, torch.int32, torch.int64, torch.uint8, torch.float8_e4m3fn
LAYOUT = {"half": e3.ROPE_HALF, "interleaved": e3.ROPE_INTERLEAVED}
SCALING = {"none": e3.ROPE_NONE, "linear": e3.ROPE_LINEAR, "base": e3.ROPE_BASE, "bands": e3.ROPE_BANDS, "ramp": e3.ROPE_RAMP}


def _np(t):
    return t.double().cpu().numpy()


def _table(dev, R, scaling="none", theta=500000.0):
    t = torch.full((R // 2,), -1, dtype=i64, device=dev)
    high = 32.0 if scaling == "ramp" else 4.0
    e3.eagle3_rope_table(t, theta=theta, scaling=SCALING[scaling], factor=8.0, high_turns=high, original_positions=4096)
    return t, kv.frequencies(R, theta, scaling, 8.0, 1.0, high, 4096)


# ----------------------------------------------------------------------------- rotations
@pytest.mark.parametrize("scaling", list(SCALING))
@pytest.mark.parametrize("R", [4, 20, 64, 128, 256])
def test_rope_table(R, scaling):
    dev = require_gpu()
    t, f = _table(dev, R, scaling)
    turns = [(int(v) % 2 ** 64) / 2.0 ** 64 for v in t.cpu()]
    # pow, log and the divisions of fp64: a few steps of 2^-52
    assert np.allclose(turns, f / (2 * math.pi), rtol=2.0 ** -47, atol=2.0 ** -64)


def _check_rope(T, H, D, R, layout, dtype, scaling="none", inverse=False, amplitude=1.0, pitch=0, far=5000, seed=0,
                in_place=False, positions=None):
    dev = require_gpu()
    g = torch.Generator().manual_seed(seed + T + H + D + R)
    full = torch.randn(T, H * D + pitch, generator=g).to(dtype)
    x = full.to(dev)
    pos = torch.randint(0, far, (T,), generator=g, dtype=i32) if positions is None else positions
    table, f = _table(dev, R, scaling)
    view = x[:, :H * D].unflatten(1, (H, D))
    out_full = x if in_place else torch.full((T, H * D + pitch), 7.0, dtype=dtype, device=dev)
    out = out_full[:, :H * D].unflatten(1, (H, D))
    e3.eagle3_rope(view, pos.to(dev), table, out, layout=LAYOUT[layout], inverse=inverse, amplitude=amplitude)
    torch.cuda.synchronize()
    src = full[:, :H * D].double().numpy().reshape(T, H, D)
    want = kv.rope(src, pos.numpy(), f, layout, inverse, amplitude)
    a, b = kv.pairs(R, layout)
    both = np.zeros_like(src)
    both[..., a] = both[..., b] = np.abs(src[..., a]) + np.abs(src[..., b])
    # the table's rounding, 2^-52 of a turn's fraction and 2^-65 turns, over the distance
    reach = np.abs(pos.numpy().astype(np.float64)).max() if T else 0.0
    tol = abs(amplitude) * both * (10 * U + reach * 2 * math.pi * 2.0 ** -50)
    tol += (BF16 if dtype is bf else U) * (np.abs(want) + tol)
    tol[..., R:] = 0
    err = np.abs(_np(out) - want)
    assert (err <= tol).all(), (float((err / (tol + 1e-30)).max()), float(err.max()))
    if pitch:
        assert (out_full[:, H * D:] == (x[:, H * D:] if in_place else 7)).all()
    assert in_place or torch.equal(x.cpu(), full)


@pytest.mark.parametrize("dtype", [bf, f32], ids=["bf16", "f32"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("T,H,D,R", [(1, 1, 8, 2), (1, 40, 128, 128), (3, 2, 64, 64), (2, 5, 96, 64), (7, 3, 80, 20),
                                     (65, 4, 128, 48), (300, 1, 256, 256), (33, 17, 96, 96), (5, 2, 128, 126),
                                     (2, 1, 256, 2), (1500, 6, 64, 32), (1, 600, 64, 64)])
def test_rope(T, H, D, R, layout, dtype):
    _check_rope(T, H, D, R, layout, dtype)


@pytest.mark.parametrize("dtype", [bf, f32], ids=["bf16", "f32"])
@pytest.mark.parametrize("scaling", list(SCALING))
def test_rope_scaled_far_inverse_pitched(scaling, dtype):
    _check_rope(130, 3, 128, 128, "half", dtype, scaling, far=1 << 20, pitch=64, amplitude=1.2079)
    _check_rope(130, 3, 128, 96, "interleaved", dtype, scaling, far=1 << 20, pitch=8, inverse=True, amplitude=-0.5)


@pytest.mark.parametrize("R", [128, 100])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rope_in_place(layout, R):
    _check_rope(70, 5, 128, R, layout, bf, pitch=16, in_place=True)


def test_rope_extreme_positions():
    p = torch.tensor([0, 1, -1, 2 ** 31 - 1, -2 ** 31, 2 ** 30 + 1], dtype=i32)
    _check_rope(6, 2, 64, 64, "half", f32, positions=p)


def test_rope_of_no_rows():
    _check_rope(0, 2, 64, 64, "half", f32, far=1)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rope_gradient(layout):
    """The inverse call is the gradient: against differences of the forward call, and R(t)^T R(t) = amplitude^2."""
    dev = require_gpu()
    g = torch.Generator().manual_seed(5)
    x = torch.randn(4, 2, 32, generator=g).to(dev)
    up = torch.randn(4, 2, 32, generator=g).to(dev)
    pos = torch.tensor([0, 3, 1000, 70000], dtype=i32, device=dev)
    table, _ = _table(dev, 24, "ramp")
    call = lambda v, inv: (e3.eagle3_rope(v, pos, table, o := torch.empty_like(v), layout=LAYOUT[layout], inverse=inv,
                                          amplitude=1.5), o)[1]
    grad = call(up, True)
    # the map is linear: a difference of step 1 in one element is exact but for fp32's roundings of |x| + 1
    for d in (0, 1, 11, 12, 23, 24, 31):
        step = torch.zeros_like(x)
        step[..., d] = 1
        diff = ((call(x + step, False) - call(x, False)) * up).sum(-1)
        want = grad[..., d]
        bound = 1.5 * 24 * U * ((x.abs() + 1).sum(-1) * up.abs().sum(-1))
        assert ((diff - want).abs() <= bound).all()


def test_rope_in_a_graph_and_on_another_stream():
    dev = require_gpu()
    x, pos = torch.randn(90, 4, 64, device=dev), torch.arange(90, dtype=i32, device=dev)
    table, _ = _table(dev, 64)
    out, again = torch.empty_like(x), torch.empty_like(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
        e3.eagle3_rope(x, pos, table, out)
    for shift in (0, 1000):
        pos.add_(shift)
        graph.replay()
        e3.eagle3_rope(x, pos, table, again, stream=torch.cuda.current_stream())
        torch.cuda.synchronize()
        assert torch.equal(out, again)


# ----------------------------------------------------------------------------- appends
class Pool:
    """An e4m3 pool and its oracle's copy, pages in random order."""

    def __init__(self, dev, lens, Hkv, D, size, seed, spare=2, columns=None):
        self.g = torch.Generator().manual_seed(seed)
        self.size, self.Hkv, self.D, self.dev = size, Hkv, D, dev
        need = [-(-n // size) for n in lens]
        self.pages = sum(need) + spare
        order = torch.randperm(self.pages, generator=self.g).tolist()
        cols = columns or max(1, max(need, default=1))
        self.table = np.full((len(lens), cols), -1, np.int32)
        for b, n in enumerate(need):
            self.table[b, :n] = [order.pop() for _ in range(n)]
        rnd = lambda *s: torch.randint(0, 256, s, generator=self.g, dtype=torch.int32).to(u8)
        # what is left of earlier sequences: any codes (NaN too) and any scales
        self.codes = [rnd(self.pages, Hkv, size, D) for _ in range(2)]
        self.scale = [rnd(self.pages, Hkv, size // 64) for _ in range(2)]

    def fill(self, lens, spread=1.0):
        """Sequences of these lengths by the oracle's append; returns their rows."""
        for t in range(2):
            c, s = self.codes[t].numpy(), self.scale[t].numpy()
            for b, n in enumerate(lens):
                rows = torch.randn(n, self.Hkv, self.D, generator=self.g).double().numpy() * spread
                kv.append(c, s, self.table[b].tolist(), 0, rows, self.pages)
        return self

    def device(self):
        c = [t.to(self.dev).view(f8) for t in self.codes]
        s = [t.to(self.dev) for t in self.scale]
        return c, s, torch.from_numpy(self.table).to(self.dev)


def _ints(v, dev):
    return torch.tensor(v, dtype=i32, device=dev)


def _check_append(lens, new, Hkv, D, size, R=0, layout="half", scaling="none", seed=0, amplitude=1.0, spread=1.0):
    dev = require_gpu()
    B = len(lens)
    pool = Pool(dev, [a + n for a, n in zip(lens, new)], Hkv, D, size, seed).fill(lens)
    g = torch.Generator().manual_seed(seed + 1)
    T = sum(new)
    rows = (torch.randn(T + 1, 2 * Hkv, D, generator=g) * torch.exp(spread * torch.randn(T + 1, 1, 1, generator=g))).to(bf)
    start = [sum(new[:b]) for b in range(B)]
    (kc, vc), (ks, vs), table = pool.device()
    rd = rows.to(dev)
    st = torch.zeros(1, dtype=i32, device=dev)
    rope = _table(dev, R, scaling) if R else None
    e3.eagle3_append_kv(rd[:, :Hkv], rd[:, Hkv:], _ints(lens, dev), _ints(new, dev), table, kc, vc, max_new=max(new),
                        block_size=size, k_scale=ks, v_scale=vs, row_start=_ints(start, dev),
                        rope_table=rope[0] if R else None, rope_layout=LAYOUT[layout], rope_amplitude=amplitude,
                        dev_status=st)
    torch.cuda.synchronize()
    assert int(st) == 0
    for t, (codes, scale) in enumerate(((kc, ks), (vc, vs))):
        before = pool.codes[t].numpy().copy()
        c, s = pool.codes[t].numpy(), pool.scale[t].numpy()
        src = rows[:, t * Hkv:(t + 1) * Hkv].double().numpy()
        slack = np.zeros(c.shape)
        for b in range(B):
            r = src[start[b]:start[b] + new[b]]
            if R and t == 0:
                pos = lens[b] + np.arange(new[b])
                a2, b2 = kv.pairs(R, layout)
                both = np.zeros_like(r)
                both[..., a2] = both[..., b2] = np.abs(r[..., a2]) + np.abs(r[..., b2])
                r = kv.rope(r, pos, rope[1], layout, amplitude=amplitude)
                for j in range(new[b]):
                    slack[table[b, pos[j] // size].item(), :, pos[j] % size] = abs(amplitude) * 10 * U * both[j]
            kv.append(c, s, pool.table[b].tolist(), lens[b], r, pool.pages)
        np.testing.assert_array_equal(scale.cpu().numpy(), s)
        got = codes.view(u8).cpu().numpy()
        if not (R and t == 0):
            np.testing.assert_array_equal(got & np.where(fp8.decode(c) != fp8.decode(c), 0x7F, 0xFF), c & np.where(
                fp8.decode(c) != fp8.decode(c), 0x7F, 0xFF))
            continue
        # turned keys: a code may differ from the oracle's where fp32 lands on the other side of a rounding
        same = slack == 0
        np.testing.assert_array_equal(got[same & (c != 0x7F)], c[same & (c != 0x7F)])
        f = np.repeat(2.0 ** (s.astype(np.float64) - 127), 64, 2)[..., None]
        for b in range(B):
            pos = lens[b] + np.arange(new[b])
            r = kv.rope(src[start[b]:start[b] + new[b]], pos, rope[1], layout, amplitude=amplitude)
            for j in range(new[b]):
                at = (pool.table[b, pos[j] // size], slice(None), pos[j] % size)
                err = np.abs(fp8.decode(got[at]) * f[at] - r[j])
                tol = np.maximum(np.abs(r[j]) * 2.0 ** -4, f[at] * 2.0 ** -10) + 1.07 * slack[at]
                assert (err <= tol).all(), (b, j, float((err - tol).max()))
        assert before.shape == c.shape


APPENDS = [
    ([0], [1], 1, 8, 64), ([63], [1], 2, 128, 64), ([64], [1], 2, 128, 64), ([5], [2], 3, 64, 128),
    ([60, 0, 127, 1], [8, 3, 1, 5], 2, 128, 128), ([60, 0, 10], [9, 70, 64], 2, 128, 64),
    ([0, 200], [130, 300], 3, 96, 192), ([1], [191], 1, 256, 64), ([33, 64], [31, 65], 5, 40, 256),
    ([0] * 9, [1] * 9, 8, 128, 64), ([100], [1000], 8, 128, 256)]


@pytest.mark.parametrize("lens,new,Hkv,D,size", APPENDS)
def test_append_e4m3(lens, new, Hkv, D, size):
    _check_append(lens, new, Hkv, D, size)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("lens,new,Hkv,D,size,R", [
    ([4000], [1], 2, 128, 64, 128), ([60, 0, 127], [8, 3, 1], 2, 128, 128, 128), ([33, 1000], [100, 65], 2, 96, 64, 64),
    ([0, 7], [130, 64], 1, 256, 64, 256), ([61], [5], 2, 64, 64, 20), ([0], [70], 2, 64, 64, 36), ([0], [66], 1, 80, 64, 80)])
def test_append_e4m3_turned(lens, new, Hkv, D, size, R, layout):
    _check_append(lens, new, Hkv, D, size, R, layout, "bands" if R > 20 else "none", amplitude=1.25)


def test_append_growing_and_shrinking_scales():
    """Rows of magnitudes far apart, one token at a time into groups with older ones."""
    for seed in range(4):
        _check_append([63, 62, 3, 70], [1, 1, 1, 1], 4, 64, 64, spread=6.0, seed=seed)
        _check_append([63, 62, 3, 70], [40, 9, 64, 1], 4, 64, 64, spread=6.0, seed=seed)


@pytest.mark.parametrize("D,size,lens,new,R,layout", [
    (128, 16, [0, 500, 17], [300, 1, 64], 128, "half"), (96, 17, [3, 5], [9, 130], 64, "interleaved"),
    (64, 1, [2, 0], [3, 1], 0, "half"), (128, 64, [10, 0, 63], [1, 1, 1], 60, "half")])
def test_append_bf16(D, size, lens, new, R, layout):
    dev = require_gpu()
    Hkv, B = 3, len(lens)
    g = torch.Generator().manual_seed(D)
    need = [-(-(a + n) // size) for a, n in zip(lens, new)]
    pages = sum(need) + 1
    order = torch.randperm(pages, generator=g).tolist()
    table = np.full((B, max(need)), -1, np.int32)
    for b, n in enumerate(need):
        table[b, :n] = [order.pop() for _ in range(n)]
    T = sum(new)
    rows = torch.randn(T, 2 * Hkv, D, generator=g).to(bf)
    start = [sum(new[:b]) for b in range(B)]
    pools = [torch.full((pages * size, Hkv, D), 9.0, dtype=bf, device=dev) for _ in range(2)]
    rope = _table(dev, R) if R else None
    st = torch.zeros(1, dtype=i32, device=dev)
    rd = rows.to(dev)
    e3.eagle3_append_kv(rd[:, :Hkv], rd[:, Hkv:], _ints(lens, dev), _ints(new, dev), torch.from_numpy(table).to(dev), *pools,
                        max_new=max(new), block_size=size, row_start=_ints(start, dev),
                        rope_table=rope[0] if R else None, rope_layout=LAYOUT[layout], dev_status=st)
    assert int(st) == 0
    for t in range(2):
        want, tol = np.full((pages * size, Hkv, D), 9.0), np.zeros((pages * size, Hkv, D))
        for b in range(B):
            r = rows[start[b]:start[b] + new[b], t * Hkv:(t + 1) * Hkv].double().numpy()
            pos = lens[b] + np.arange(new[b])
            slot = table[b, pos // size] * size + pos % size
            if R and t == 0:
                a2, b2 = kv.pairs(R, layout)
                both = np.zeros_like(r)
                both[..., a2] = both[..., b2] = np.abs(r[..., a2]) + np.abs(r[..., b2])
                r = kv.rope(r, pos, rope[1], layout)
                tol[slot] = np.where(both > 0, 10 * U * both + BF16 * (np.abs(r) + 10 * U * both), 0)
            want[slot] = r
        assert (np.abs(_np(pools[t]) - want) <= tol).all()


def test_append_row_ids_padded_rows_and_non_finite_values():
    dev = require_gpu()
    B, N, W, Hkv, D = 3, 6, 4, 2, 64
    lens = [62, 0, 64]
    path = [[0, 2, 5, -1], [3, -1, 1, 1], [0, 1, 1, 4]]        # ends at the first -1; a node may come twice
    counts = [3, 1, 4]
    g = torch.Generator().manual_seed(3)
    tree = torch.randn(B, N, 2 * Hkv, D, generator=g).to(bf)
    tree[0, 2, 1, 5], tree[2, 4, 0, 7], tree[2, 4, 3, 1] = float("inf"), float("nan"), -float("inf")
    for how in ("path", "path and counts", "padded"):
        pool = Pool(dev, [n + W for n in lens], Hkv, D, 64, 8).fill(lens)
        (kc, vc), (ks, vs), table = pool.device()
        if how == "padded":
            rows = torch.stack([tree[b, [max(0, i) for i in path[b]]] for b in range(B)]).reshape(B * W, 2 * Hkv, D).to(dev)
            kw = dict(n_new=_ints(counts, dev))
        else:
            rows = tree.reshape(B * N, 2 * Hkv, D).to(dev)
            kw = dict(row_ids=_ints(path, dev), rows_per_seq=N, n_new=None if how == "path" else _ints(counts, dev))
        n_new = kw.pop("n_new")
        st = torch.zeros(1, dtype=i32, device=dev)
        e3.eagle3_append_kv(rows[:, :Hkv], rows[:, Hkv:], _ints(lens, dev), n_new, table, kc, vc, max_new=W, block_size=64,
                            k_scale=ks, v_scale=vs, dev_status=st, **kw)
        assert int(st) == 0
        for t, (codes, scale) in enumerate(((kc, ks), (vc, vs))):
            c, s = pool.codes[t].numpy(), pool.scale[t].numpy()
            nan_before = np.isnan(fp8.decode(c))
            for b in range(B):
                r = tree[b, path[b][:counts[b]], t * Hkv:(t + 1) * Hkv].double().numpy()
                kv.append(c, s, pool.table[b].tolist(), lens[b], r, pool.pages)
            np.testing.assert_array_equal(scale.cpu().numpy(), s)
            got = codes.view(u8).cpu().numpy()
            nan = np.isnan(fp8.decode(c))
            np.testing.assert_array_equal(np.isnan(fp8.decode(got)), nan)
            np.testing.assert_array_equal(got[~nan], c[~nan])
            assert nan.sum() - nan_before.sum() != 0


@pytest.mark.parametrize("many", [False, True])
def test_append_leaves_out_what_is_wrong(many):
    """Counts, lengths, pages and rows out of range: flagged and left out, everything else as it would be."""
    dev = require_gpu()
    Hkv, D, size, W = 2, 64, 64, 70 if many else 4
    lens = [0, 10, -1, 126, 5, 7, 60, 3]
    new = [W, W + 1, 1, 3, -1, 2, 4, 0]
    pool = Pool(dev, [128] * 8, Hkv, D, size, 4).fill([max(0, n) for n in lens])
    pool.table[5, 0] = pool.pages      # a page that is not in the pool
    pool.table[6, 1] = -3              # the second group's page
    g = torch.Generator().manual_seed(4)
    rows = torch.randn(8 * W, 2 * Hkv, D, generator=g).to(bf)
    start = [b * W for b in range(8)]
    start[0] = 8 * W - 2               # runs past the rows: two tokens only
    st = torch.zeros(1, dtype=i32, device=dev)
    (kc, vc), (ks, vs), table = pool.device()
    rd = rows.to(dev)
    e3.eagle3_append_kv(rd[:, :Hkv], rd[:, Hkv:], _ints(lens, dev), _ints(new, dev), table, kc, vc, max_new=W,
                        block_size=size, k_scale=ks, v_scale=vs, row_start=_ints(start, dev), dev_status=st)
    assert int(st) == (0x2 | 0x4)
    for t, (codes, scale) in enumerate(((kc, ks), (vc, vs))):
        c, s = pool.codes[t].numpy(), pool.scale[t].numpy()
        r = rows[:, t * Hkv:(t + 1) * Hkv].double().numpy()
        kv.append(c, s, pool.table[0].tolist(), 0, r[start[0]:start[0] + 2], pool.pages)
        if many:   # the second group of the sequence has no row at all: its scale is that of nothing
            s[pool.table[0, 1], :, 0] = 1
        kv.append(c, s, pool.table[6].tolist(), 60, r[start[6]:start[6] + 4], pool.pages)
        np.testing.assert_array_equal(scale.cpu().numpy(), s)
        got, nan = codes.view(u8).cpu().numpy(), np.isnan(fp8.decode(c))
        np.testing.assert_array_equal(got[~nan], c[~nan])
        np.testing.assert_array_equal(np.isnan(fp8.decode(got)), nan)


def test_append_offsets_past_32_bits():
    """The last pages of a pool of more than 2^32 codes."""
    dev = require_gpu()
    Hkv, D, size = 8, 128, 256
    pages = (1 << 32) // (Hkv * D * size) + 2
    kc, vc = (torch.zeros(pages, Hkv, size, D, dtype=u8, device=dev) for _ in range(2))
    ks, vs = (torch.zeros(pages, Hkv, size // 64, dtype=u8, device=dev) for _ in range(2))
    rows = torch.randn(70, 2 * Hkv, D, generator=torch.Generator().manual_seed(1)).to(bf)
    table = np.array([[pages - 1]], np.int32)
    rd = rows.to(dev)
    e3.eagle3_append_kv(rd[:, :Hkv], rd[:, Hkv:], _ints([0], dev), _ints([70], dev), torch.from_numpy(table).to(dev),
                        kc.view(f8), vc.view(f8), max_new=70, block_size=size, k_scale=ks, v_scale=vs,
                        row_start=_ints([0], dev))
    c, s = np.zeros((1, Hkv, size, D), np.uint8), np.zeros((1, Hkv, 4), np.uint8)
    kv.append(c, s, [0], 0, rows[:, :Hkv].double().numpy(), 1)
    np.testing.assert_array_equal(kc[-1].cpu().numpy(), c[0])
    np.testing.assert_array_equal(ks[-1].cpu().numpy(), s[0])
    assert int(kc[:-1].max()) == 0 and int(vc[:-1].max()) == 0


# ----------------------------------------------------------------------------- attention
def pytest_generate_tests(metafunc):
    """Each attention test by the kernel that the call chooses and, where it takes the call, by the one of 128 rows."""
    if metafunc.function.__name__.startswith("test_attn"):
        metafunc.parametrize("kernel", ["own choice", "128 rows"], indirect=True)


@pytest.fixture(autouse=True)
def kernel(request, monkeypatch):
    if getattr(request, "param", None) != "128 rows":
        return
    public = e3.eagle3_verify_attn_fp8

    def call(q, k_cache, *args, **kw):
        if q.shape[1] * q.shape[2] // k_cache.shape[1] <= 16:
            return public(q, k_cache, *args, **kw)
        return _lib.eagle3_test_verify_attn_fp8(q, k_cache, *args, kernel=2, **kw)
    monkeypatch.setattr(e3, "eagle3_verify_attn_fp8", call)


def _trees(B, N, seed):
    r = np.random.default_rng(seed)
    par = np.full((B, N), -1, np.int32)
    for i in range(1, N):
        par[:, i] = r.integers(max(0, i - 9), i, B)
    return par


def _attn_inputs(dev, lens, N, Hq, Hkv, size, seed, tree, q_spread=1.5, columns=None):
    pool = Pool(dev, lens, Hkv, 128, size, seed, columns=columns).fill(lens)
    g = torch.Generator().manual_seed(seed + 7)
    B = len(lens)
    q = (q_spread * torch.randn(B, N, Hq, 128, generator=g)).to(bf)
    tk = torch.randn(B, N, Hkv, 128, generator=g).to(bf) if tree else None
    tv = torch.randn(B, N, Hkv, 128, generator=g).to(bf) if tree else None
    return pool, q, tk, tv, _trees(B, N, seed) if tree else None


def _expected(pool, lens, q, tk, tv, par, sm_scale=0.0):
    outs = []
    for b, n in enumerate(lens):
        k = kv.read(pool.codes[0].numpy(), pool.scale[0].numpy(), pool.table[b].tolist(), n, pool.pages)
        v = kv.read(pool.codes[1].numpy(), pool.scale[1].numpy(), pool.table[b].tolist(), n, pool.pages)
        t = (tk[b].double().numpy(), tv[b].double().numpy(), par[b].tolist()) if tk is not None else (None, None, None)
        qb = q[b].double().numpy()
        out, lse, mag, dot = kv.attention(qb, k, v, *t, sm_scale=sm_scale)
        ks = [np.abs(k).sum(2).max() if n else 0.0, np.abs(t[0]).sum(2).max() if tk is not None else 0.0]
        vs = [np.abs(v).max() if n else 0.0, np.abs(t[1]).max() if tk is not None else 0.0]
        keys = n + (q.shape[1] if tk is not None else 0)
        parts = np.abs(qb).max(2) * max(ks) + (np.abs(t[0]).max() * np.abs(qb).sum(2) if tk is not None else 0.0)
        w = 262 * U * dot + 2.0 ** -17 * parts * (sm_scale or 128 ** -0.5) + 2.0 ** -21
        acc = (keys + 64) * 2 * U
        tol = (2 * w + 2.0 ** -11 + acc)[..., None] * mag + keys * 2.0 ** -31 * max(vs)
        tol = tol + BF16 * (np.abs(out) + tol)
        lse_tol = w + acc + 8 * U * np.abs(np.where(np.isfinite(lse), lse, 0.0))
        outs.append((out, lse, tol, lse_tol))
    return [np.stack(x) for x in zip(*outs)]


def _call(pool, lens, q, tk, tv, par, dev, longest=None, **kw):
    (kc, vc), (ks, vs), table = pool.device()
    B, N, Hq, D = q.shape
    out = torch.full((B, N, Hq, D), 7.0, dtype=bf, device=dev)
    lse = torch.full((B, N, Hq), 7.0, device=dev)
    st = torch.zeros(1, dtype=i32, device=dev)
    t = lambda x: None if x is None else (x if isinstance(x, torch.Tensor) else torch.from_numpy(x)).to(dev)
    e3.eagle3_verify_attn_fp8(q.to(dev), kc, vc, ks, vs, table, _ints(lens, dev), out,
                              max_prefix_len=max(lens) if longest is None else longest, tree_k=t(tk), tree_v=t(tv),
                              parents=t(par), lse=lse, dev_status=st, **kw)
    torch.cuda.synchronize()
    return out, lse, int(st)


def _check_attn(lens, N, Hq, Hkv, size, tree, seed=0, sm_scale=0.0, longest=None, q_spread=1.5, **kw):
    dev = require_gpu()
    pool, q, tk, tv, par = _attn_inputs(dev, lens, N, Hq, Hkv, size, seed, tree, q_spread,
                                        columns=None if longest is None else -(-longest // size))
    out, lse, st = _call(pool, lens, q, tk, tv, par, dev, longest, sm_scale=sm_scale, **kw)
    assert st == 0
    want, want_lse, tol, lse_tol = _expected(pool, lens, q, tk, tv, par, sm_scale)
    err = np.abs(_np(out) - want)
    assert (err <= tol).all(), (float((err / tol).max()), float(err.max()))
    empty = np.isinf(want_lse)
    got = _np(lse)
    assert (got[empty] == -np.inf).all()
    assert (np.abs(got[~empty] - want_lse[~empty]) <= lse_tol[~empty]).all()


SINGLE = [([1], 1, 1, 1, 64), ([0], 1, 4, 1, 64), ([31, 32, 33], 1, 8, 2, 64), ([63, 64, 65, 0], 1, 8, 2, 128),
          ([700], 1, 32, 8, 64), ([129, 1], 1, 16, 1, 192), ([300, 5], 1, 17, 1, 64), ([100], 3, 4, 4, 64),
          ([200, 90], 2, 48, 3, 256), ([2000, 1, 999], 1, 32, 8, 256)]


@pytest.mark.parametrize("lens,N,Hq,Hkv,size", SINGLE)
def test_attn_single_tokens(lens, N, Hq, Hkv, size):
    _check_attn(lens, N, Hq, Hkv, size, False)


@pytest.mark.parametrize("lens,N,Hq,Hkv,size", [
    ([0], 1, 1, 1, 64), ([0, 5], 4, 8, 2, 64), ([64, 1], 17, 4, 1, 64), ([65, 130, 0], 9, 6, 2, 64),
    ([127, 300], 32, 4, 1, 128), ([200, 0, 128], 60, 8, 2, 128), ([333], 64, 12, 3, 192), ([100, 257], 64, 8, 1, 256),
    ([70], 64, 16, 1, 64), ([513, 12], 33, 32, 8, 64), ([400], 3, 44, 1, 64)])
def test_attn_trees(lens, N, Hq, Hkv, size):
    _check_attn(lens, N, Hq, Hkv, size, True)


@pytest.mark.parametrize("splits", [1, 2, 3, 7, 64])
@pytest.mark.parametrize("N,Hq,tree", [(1, 8, False), (5, 8, True), (60, 8, True)])
def test_attn_splits(N, Hq, tree, splits):
    _check_attn([500, 31, 0, 170], N, Hq, 2, 64, tree, num_splits=splits)


@pytest.mark.parametrize("lens,N,Hq,splits", [([3000, 40], 1, 8, 47), ([3000, 0], 3, 16, 33), ([1500, 600], 5, 8, 12), ([20000], 1, 8, 2000),
                                              ([2500] * 40, 1, 8, 3), ([2500, 9] * 20, 3, 16, 8), ([1000], 1, 8, 5)])
def test_attn_many_parts(lens, N, Hq, splits):
    """Parts of few steps, joined by a warp or a CTA a row or within a cluster; more parts asked for than there are."""
    _check_attn(lens, N, Hq, 2, 64, N > 1, num_splits=splits)


@pytest.mark.parametrize("B,splits", [(1, 3), (1, 8), (2, 20), (40, 4)])
def test_attn_nan_in_one_part(B, splits):
    """A NaN key or value in one of many parts reaches its sequence's rows of that KV head, and no others."""
    dev = require_gpu()
    lens = [1500] * B
    pool, q, tk, tv, par = _attn_inputs(dev, lens, 1, 8, 2, 64, 13, False)
    pool.codes[0].numpy()[pool.table[0, 11], 0, 9, 3] = 0x7F
    pool.codes[1].numpy()[pool.table[B - 1, 20], 1, 9, 5] = 0xFF
    out, _, st = _call(pool, lens, q, tk, tv, par, dev, num_splits=splits)
    nan = torch.isnan(out).cpu().numpy()
    want = np.zeros(nan.shape, bool)
    want[0, :, :4] = True
    want[B - 1, :, 4:, 5] = True
    assert st == 0
    np.testing.assert_array_equal(nan, want)


@pytest.mark.parametrize("lens,N,Hq", [([12000, 3], 5, 8), ([9000], 33, 4), ([5000, 7000, 0, 130], 60, 4)])
def test_attn_many_tiles_in_a_row(lens, N, Hq):
    """Hundreds of tiles for one CTA: every ring and barrier goes around many times."""
    _check_attn(lens, N, Hq, 1, 128, True, num_splits=1)


def test_attn_full_gpu_repeats():
    """Every SM busy over many units: bit-identical every time, and equal to the oracle for two sequences."""
    dev = require_gpu()
    B, N, Hq, Hkv, L, size = 48, 60, 32, 8, 1500, 128
    lens = [L - 17 * b for b in range(B)]
    g = torch.Generator(device=dev).manual_seed(3)
    need = [-(-n // size) for n in lens]
    pages = sum(need)
    ids = torch.randperm(pages, generator=g, device=dev).to(i32)
    table = torch.full((B, max(need)), -1, dtype=i32, device=dev)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = ids[at:at + n]
        at += n
    caches = [torch.randn(pages, Hkv, size, 128, generator=g, device=dev).mul_(60).to(f8) for _ in range(2)]
    scales = [torch.randint(119, 122, (pages, Hkv, size // 64), generator=g, device=dev, dtype=i32).to(u8) for _ in range(2)]
    q, tk, tv = (torch.randn(B, N, h, 128, generator=g, device=dev).to(bf) for h in (Hq, Hkv, Hkv))
    par = _trees(B, N, 5)
    st = torch.zeros(1, dtype=i32, device=dev)
    outs = [torch.empty(B, N, Hq, 128, dtype=bf, device=dev) for _ in range(2)]
    for i in range(60):
        e3.eagle3_verify_attn_fp8(q, *caches, *scales, table, _ints(lens, dev), outs[min(i, 1)], max_prefix_len=L, tree_k=tk,
                                  tree_v=tv, parents=torch.from_numpy(par).to(dev), dev_status=st)
        assert i == 0 or torch.equal(outs[0], outs[1])
    assert int(st) == 0
    pool = Pool(dev, [64], Hkv, 128, size, 1)
    pool.pages = pages
    pool.codes = [c.view(u8).cpu() for c in caches]
    pool.scale = [c.cpu() for c in scales]
    for b in (0, B - 1):
        pool.table = table[b:b + 1].cpu().numpy()
        want, _, tol, _ = _expected(pool, lens[b:b + 1], q[b:b + 1].cpu(), tk[b:b + 1].cpu(), tv[b:b + 1].cpu(), par[b:b + 1])
        assert (np.abs(_np(outs[0][b:b + 1]) - want) <= tol).all()


@pytest.mark.parametrize("N,Hq", [(1, 8), (60, 8)])
def test_attn_bound_above_the_lengths(N, Hq):
    _check_attn([200, 0, 1], N, Hq, 2, 64, N > 1, longest=3000)


@pytest.mark.parametrize("N,Hq", [(1, 8), (60, 8)])
def test_attn_scales_of_scores(N, Hq):
    _check_attn([150, 70], N, Hq, 2, 64, N > 1, sm_scale=0.3, seed=1)      # sharp weights
    _check_attn([150, 70], N, Hq, 2, 64, N > 1, sm_scale=1e-6, seed=2)     # flat ones
    _check_attn([150, 70], N, Hq, 2, 64, N > 1, q_spread=0.0, seed=3)      # queries of zero
    _check_attn([150, 70], N, Hq, 2, 64, N > 1, q_spread=1e5, sm_scale=1e-5, seed=4)
    _check_attn([150, 70], N, Hq, 2, 64, N > 1, q_spread=1e-30, sm_scale=1e28, seed=5)


@pytest.mark.parametrize("N,Hq", [(1, 8), (60, 8)])
def test_attn_groups_of_unlike_scales(N, Hq):
    """K and V of each group by a factor of its own, groups of zeros among them, growing and falling."""
    dev = require_gpu()
    lens = [400, 130]
    for seed in range(3):
        pool, q, tk, tv, par = _attn_inputs(dev, lens, N, Hq, 2, 64, seed, N > 1, q_spread=0.3)
        r = np.random.default_rng(seed)
        s = pool.scale[1].numpy()
        s[:] = np.clip(s.astype(int) + r.integers(-9, 10, s.shape), 1, 254)
        pool.scale[0].numpy()[:] = np.clip(pool.scale[0].numpy().astype(int) + r.integers(-3, 2, s.shape), 1, 254)
        for t in range(2):
            pool.codes[t].numpy()[pool.table[0, 2], 0] = 0          # a group of zeros, as an append writes it
            pool.scale[t].numpy()[pool.table[0, 2], 0] = 1
        out, _, st = _call(pool, lens, q, tk, tv, par, dev)
        want, _, tol, _ = _expected(pool, lens, q, tk, tv, par)
        assert st == 0 and (np.abs(_np(out) - want) <= tol).all()


@pytest.mark.parametrize("N,Hq", [(1, 8), (60, 8)])
def test_attn_does_not_look_past_the_lengths(N, Hq):
    """NaN codes and scales behind every sequence's last position, and in groups that no sequence has reached."""
    dev = require_gpu()
    lens = [70, 64, 1, 0]
    pool, q, tk, tv, par = _attn_inputs(dev, lens, N, Hq, 2, 128, 6, N > 1)
    for t in range(2):
        c, s = pool.codes[t].numpy(), pool.scale[t].numpy()
        used = np.zeros(c.shape[:3], bool)
        for b, n in enumerate(lens):
            for p in range(n):
                used[pool.table[b, p // 128], :, p % 128] = True
        c[~used] = 0x7F
        s[~used.reshape(*s.shape, 64).any(3)] = 255
    out, lse, st = _call(pool, lens, q, tk, tv, par, dev)
    want, want_lse, tol, _ = _expected(pool, lens, q, tk, tv, par)
    assert st == 0 and (np.abs(_np(out) - want) <= tol).all()
    assert (torch.isfinite(lse).cpu().numpy() == np.isfinite(want_lse)).all()


@pytest.mark.parametrize("N,Hq", [(1, 8), (60, 8)])
def test_attn_nan_before_the_length(N, Hq):
    """A NaN key makes its sequence's rows of that KV head NaN; a NaN value the dims it is in."""
    dev = require_gpu()
    lens = [200, 90]
    pool, q, tk, tv, par = _attn_inputs(dev, lens, N, Hq, 2, 64, 7, N > 1)
    pool.codes[0].numpy()[pool.table[0, 1], 0, 9, 3] = 0x7F
    pool.codes[1].numpy()[pool.table[1, 1], 1, 9, 5] = 0xFF
    out, _, st = _call(pool, lens, q, tk, tv, par, dev)
    nan = torch.isnan(out).cpu().numpy()
    want = np.zeros(nan.shape, bool)
    want[0, :, :Hq // 2] = True
    want[1, :, Hq // 2:, 5] = True
    assert st == 0
    np.testing.assert_array_equal(nan, want)
    pool.codes[0].numpy()[pool.table[0, 1], 0, 9, 3] = 0
    pool.codes[1].numpy()[pool.table[1, 1], 1, 9, 5] = 0
    pool.scale[0].numpy()[pool.table[0, 2], 1, 0] = 255
    pool.scale[1].numpy()[pool.table[1, 0], 0, 0] = 255
    out, _, st = _call(pool, lens, q, tk, tv, par, dev)
    nan = torch.isnan(out).cpu().numpy()
    assert st == 0 and nan[0, :, Hq // 2:].all() and nan[1, :, :Hq // 2].all()
    assert not nan[0, :, :Hq // 2].any() and not nan[1, :, Hq // 2:].any()


@pytest.mark.parametrize("N,Hq", [(5, 8), (60, 8)])
def test_attn_non_finite_tree_nodes_stay_on_their_paths(N, Hq):
    """A NaN key or value of a tree node reaches the node and its descendants, no other query."""
    dev = require_gpu()
    lens = [100, 70, 0]
    pool, q, tk, tv, par = _attn_inputs(dev, lens, N, Hq, 2, 64, 8, True)
    tk[0, 2, 0, 3] = float("nan")
    tv[1, 3, 1, 7] = float("nan")
    tv[2, 1, 0, 9] = float("inf")
    out, _, st = _call(pool, lens, q, tk, tv, par, dev)
    got = ~torch.isfinite(out).cpu().numpy()
    want = np.zeros(got.shape, bool)
    for i in range(N):
        want[0, i, :Hq // 2] = 2 in kv.path(par[0], i)
        want[1, i, Hq // 2:, 7] = 3 in kv.path(par[1], i)
        want[2, i, :Hq // 2, 9] = 1 in kv.path(par[2], i)
    assert st == 0
    np.testing.assert_array_equal(got, want)


@pytest.mark.parametrize("N,Hq", [(1, 8), (60, 8)])
def test_attn_flags(N, Hq):
    """Lengths past the bound are cut, pages outside the pool read as zeros, trees that are none end where they break."""
    dev = require_gpu()
    lens = [300, 200, 150]
    pool, q, tk, tv, par = _attn_inputs(dev, lens, N, Hq, 2, 64, 9, N > 1)
    given, lens[0] = [300, -4, 150], 200
    lens[1] = 0
    pool.table[2, 1] = pool.pages
    if N > 1:
        par[2, 4] = 9
    out, _, st = _call(pool, given, q, tk, tv, par, dev, longest=200)
    want, _, tol, _ = _expected(pool, lens, q, tk, tv, par)
    assert st == (0x4 | (0x1 if N > 1 else 0))
    assert (np.abs(_np(out) - want) <= tol).all()


@pytest.mark.parametrize("N,Hq", [(1, 8), (7, 8), (60, 8)])
def test_attn_node_strided_views(N, Hq):
    dev = require_gpu()
    lens = [100, 64]
    pool, q, tk, tv, par = _attn_inputs(dev, lens, N, Hq, 2, 64, 10, True)
    fused = torch.cat([q.flatten(2), tk.flatten(2), tv.flatten(2), torch.full((2, N, 24), float("nan"), dtype=bf)], 2).to(dev)
    a, b, c = Hq * 128, (Hq + 2) * 128, (Hq + 4) * 128
    views = [fused[..., lo:hi].unflatten(2, (-1, 128)) for lo, hi in ((0, a), (a, b), (b, c))]
    out, _, st = _call(pool, lens, *views, par, dev)
    want, _, tol, _ = _expected(pool, lens, q, tk, tv, par)
    assert st == 0 and (np.abs(_np(out) - want) <= tol).all()


@pytest.mark.parametrize("N,Hq,lens", [(1, 32, [3000, 100]), (60, 32, [700, 0])])
def test_attn_repeats_and_two_streams(N, Hq, lens):
    """Bit-identical from run to run, in a captured graph, and with two calls in flight at once."""
    dev = require_gpu()
    pool, q, tk, tv, par = _attn_inputs(dev, lens, N, Hq, 8, 64, 11, N > 1)
    (kc, vc), (ks, vs), table = pool.device()
    t = lambda x: None if x is None else (x if isinstance(x, torch.Tensor) else torch.from_numpy(x)).to(dev)
    qd, tkd, tvd, pd, L = q.to(dev), t(tk), t(tv), t(par), _ints(lens, dev)
    outs = [torch.empty(*q.shape, dtype=bf, device=dev) for _ in range(4)]

    def call(o):
        e3.eagle3_verify_attn_fp8(qd, kc, vc, ks, vs, table, L, o, max_prefix_len=max(lens), tree_k=tkd, tree_v=tvd,
                                  parents=pd)
    call(outs[0])
    side = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for s, o in zip(side, outs[1:]):
        with torch.cuda.stream(s):
            call(o)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side[0]), torch.cuda.graph(graph, stream=side[0]):
        call(outs[3])
    graph.replay()
    torch.cuda.synchronize()
    for o in outs[1:]:
        assert torch.equal(o, outs[0])


def test_attn_offsets_past_32_bits():
    """Keys on the last pages of a pool of more than 2^32 codes."""
    dev = require_gpu()
    Hkv, size = 8, 256
    pages = (1 << 32) // (Hkv * 128 * size) + 2
    small = Pool(dev, [300], Hkv, 128, size, 12, spare=0).fill([300])
    kc, vc = (torch.zeros(pages, Hkv, size, 128, dtype=u8, device=dev) for _ in range(2))
    ks, vs = (torch.zeros(pages, Hkv, size // 64, dtype=u8, device=dev) for _ in range(2))
    for t, (c, s) in enumerate(((kc, ks), (vc, vs))):
        c[-2:], s[-2:] = small.codes[t].to(dev), small.scale[t].to(dev)
    table = torch.from_numpy(small.table + (pages - 2)).to(dev)
    for N, Hq in ((1, 8), (40, 32)):
        q = torch.randn(1, N, Hq, 128, generator=torch.Generator().manual_seed(1)).to(bf)
        out = torch.empty(1, N, Hq, 128, dtype=bf, device=dev)
        e3.eagle3_verify_attn_fp8(q.to(dev), kc.view(f8), vc.view(f8), ks, vs, table, _ints([300], dev), out,
                                  max_prefix_len=300)
        want, _, tol, _ = _expected(small, [300], q, None, None, None)
        assert (np.abs(_np(out) - want) <= tol).all()


# ----------------------------------------------------------------------------- together
def test_prompt_then_tokens_then_a_tree():
    """A serving run: a ragged prompt, two single tokens and an accepted path appended, each step's attention against
    the oracle's on the codes that the cache then holds, eager and in one captured graph."""
    dev = require_gpu()
    B, Hq, Hkv, D, size, W, N = 3, 8, 2, 128, 64, 5, 12
    prompt = [70, 1, 129]
    g = torch.Generator().manual_seed(20)
    table_r, freq = _table(dev, D, "bands")
    qkv = torch.randn(4, B * N, (Hq + 2 * Hkv) * D, generator=g).to(bf).to(dev)
    big = torch.randn(sum(prompt), 2 * Hkv, D, generator=g).to(bf).to(dev)
    par = _trees(B, N, 20)
    path = [[0, 1, -1, -1, -1], [0, -1, -1, -1, -1], [0, 1, 2, 3, 4]]
    pool = Pool(dev, [200] * B, Hkv, D, size, 21)
    (kc, vc), (ks, vs), table = pool.device()
    L, st = _ints(prompt, dev), torch.zeros(1, dtype=i32, device=dev)
    zero, one = _ints([0] * B, dev), _ints([1] * B, dev)
    start = _ints([0, 70, 71], dev)
    cache = dict(block_size=size, k_scale=ks, v_scale=vs, dev_status=st)
    e3.eagle3_append_kv(big[:, :Hkv], big[:, Hkv:], zero, L, table, kc, vc, max_new=129, row_start=start,
                        rope_table=table_r, **cache)
    outs = [torch.empty(B, 1, Hq, D, dtype=bf, device=dev) for _ in range(2)]
    tree_out = torch.empty(B, N, Hq, D, dtype=bf, device=dev)
    rot = [torch.empty(B, Hq, D, dtype=bf, device=dev) for _ in range(2)]
    tree_rot = torch.empty(B * N, (Hq + Hkv), D, dtype=bf, device=dev)
    pd = torch.from_numpy(par).to(dev)
    depth = _ints([[len(kv.path(par[b], i)) - 1 for i in range(N)] for b in range(B)], dev)
    pid = _ints(path, dev)
    snaps = []

    def steps():
        for i in range(2):   # a single token: its key appended, then attended to with the rest
            row = qkv[i, :B].view(B, Hq + 2 * Hkv, D)
            e3.eagle3_rope(row[:, :Hq], L, table_r, rot[i])
            e3.eagle3_append_kv(row[:, Hq:Hq + Hkv], row[:, Hq + Hkv:], L, one, table, kc, vc, max_new=1, rope_table=table_r,
                                **cache)
            L.add_(1)
            e3.eagle3_verify_attn_fp8(rot[i].view(B, 1, Hq, D), kc, vc, ks, vs, table, L, outs[i], max_prefix_len=190,
                                      dev_status=st)
        row = qkv[2].view(B * N, Hq + 2 * Hkv, D)
        e3.eagle3_rope(row[:, :Hq + Hkv], (L[:, None] + depth).view(-1), table_r, tree_rot)
        tree = tree_rot.view(B, N, Hq + Hkv, D)
        tv = row[:, Hq + Hkv:]
        packed = torch.cat([tree_rot[:, Hq:], tv], 1)    # keys and values at one pitch
        pk = packed.view(B, N, 2 * Hkv, D)
        e3.eagle3_verify_attn_fp8(tree[:, :, :Hq], kc, vc, ks, vs, table, L, tree_out, max_prefix_len=190,
                                  tree_k=pk[:, :, :Hkv], tree_v=pk[:, :, Hkv:], parents=pd, dev_status=st)
        snaps[:] = [packed]
        e3.eagle3_append_kv(packed[:, :Hkv], packed[:, Hkv:], L, None, table, kc, vc, max_new=W, row_ids=pid, rows_per_seq=N,
                            **cache)

    saved = [t.clone() for t in (kc.view(u8), vc.view(u8), ks, vs)]
    results = []
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    for how in ("eager", "graph"):
        for t, s in zip((kc.view(u8), vc.view(u8), ks, vs), saved):
            t.copy_(s)
        L.copy_(_ints(prompt, dev))
        torch.cuda.synchronize()
        if how == "eager":
            steps()
        else:
            with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
                steps()
            graph.replay()
        torch.cuda.synchronize()
        results.append([t.clone() for t in (*outs, tree_out, kc.view(u8), vc.view(u8), ks, vs)])
    assert int(st) == 0
    for a, b in zip(*results):
        assert torch.equal(a.view(u8) if a.dtype is not u8 else a, b.view(u8) if b.dtype is not u8 else b)
    # the oracle's cache, filled the same way from the same rows
    for t in range(2):
        c, s = pool.codes[t].numpy(), pool.scale[t].numpy()
        for b in range(B):
            at = [0, 70, 71][b]
            new = [big[at:at + prompt[b], t * Hkv:(t + 1) * Hkv]]
            new += [qkv[i, b].view(-1, D)[None, Hq + t * Hkv:Hq + (t + 1) * Hkv] for i in range(2)]
            rows = np.concatenate([_np(x) for x in new])
            if t == 0:
                rows = kv.rope(rows, np.arange(len(rows)), freq)
            kv.append(c, s, pool.table[b].tolist(), 0, rows, pool.pages)
            ids = [i for i in path[b] if i >= 0]
            kv.append(c, s, pool.table[b].tolist(), len(rows),
                      _np(snaps[0].view(B, N, 2 * Hkv, D)[b, ids, t * Hkv:(t + 1) * Hkv]), pool.pages)
        got = (kc, vc)[t].view(u8).cpu().numpy()
        np.testing.assert_array_equal((ks, vs)[t].cpu().numpy(), s)
        if t == 1:
            ok = ~np.isnan(fp8.decode(c))
            np.testing.assert_array_equal(got[ok], c[ok])
        else:   # turned in fp32: a code in some thousands rounds the other way
            used = ~np.isnan(fp8.decode(c))
            f = np.repeat(2.0 ** (s.astype(np.float64) - 127), 64, 2)[..., None] * np.ones(c.shape)
            a, b = fp8.decode(got) * f, fp8.decode(c) * f
            assert (np.abs(a - b)[used] <= np.maximum(np.abs(b) * 2.0 ** -2.9, f * 2.0 ** -9)[used]).all()
            assert (got != c)[used].mean() < 1e-3
        pool.codes[t].numpy()[:] = got
    want, _, tol, _ = _expected(pool, [n + 2 for n in prompt], _cpu(tree_rot.view(B, N, -1, D)[:, :, :Hq]),
                                _cpu(snaps[0].view(B, N, -1, D)[:, :, :Hkv]), _cpu(snaps[0].view(B, N, -1, D)[:, :, Hkv:]), par)
    assert (np.abs(_np(tree_out) - want) <= tol).all()
    want, _, tol, _ = _expected(pool, [n + 2 for n in prompt], _cpu(rot[1].view(B, 1, Hq, D)), None, None, None)
    assert (np.abs(_np(outs[1]) - want) <= tol).all()


def _cpu(t):
    return t.cpu()
