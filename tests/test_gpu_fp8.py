"""GPU numerics of the 8-bit operators against the fp64 oracle.

Tolerances, from the arithmetic (u = 2^-24, half an fp32 step): quantisation is two IEEE divisions
and a conversion, so scales and codes are exact.  In the product the e4m3 products are exact; each of
the at most 128 additions of a block is off by at most one fp32 step (2 u) of a partial sum, the
scaling by 3 roundings a block, and the blocks' sum by one rounding a block: (256 + 3 + blocks) u S with
S = sum |scale products| |x| |w|.  bf16 outputs add 2^-8 of their value, SwiGLU as in the bf16 tests.
"""
import numpy as np
import pytest
import torch

import eagle_tree_speculative_spec_gb300 as e3
from oracle import fp8, moe
from tests._util import require_gpu

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF16 = 2.0 ** -8
bf, f32, i32, f8 = torch.bfloat16, torch.float32, torch.int32, torch.float8_e4m3fn


def _np(t):
    return t.double().cpu().numpy()


# ----------------------------------------------------------------------------- quantisation
def _check_quantize(x, pitch=0):
    dev = require_gpu()
    m, k = x.shape
    xd = torch.zeros(m, k + pitch, dtype=bf, device=dev)
    xd[:, :k] = x.to(dev)
    q = torch.zeros(m, k + pitch, dtype=torch.uint8, device=dev)
    scale = torch.full((-(-k // 128), m), 7.0, device=dev)
    e3.eagle3_quantize_fp8(xd[:, :k], q.view(f8)[:, :k], scale)
    torch.cuda.synchronize()
    codes, want = fp8.quantize(x.float().numpy())
    np.testing.assert_array_equal(scale.cpu().numpy(), want)
    got = q.cpu().numpy()
    nan = codes == 0x7F
    np.testing.assert_array_equal(np.where(nan, got[:, :k] & 0x7F, got[:, :k]), codes)   # a NaN's sign is free
    assert (got[:, k:] == 0).all()


@pytest.mark.parametrize("m,k,pitch", [(1, 16, 0), (1, 4096, 0), (3, 128, 0), (7, 144, 0), (64, 400, 16), (33, 1040, 0),
                                       (130, 4096, 32), (1500, 2064, 0)])
def test_quantize(m, k, pitch):
    g = torch.Generator().manual_seed(m + k)
    x = torch.randn(m, k, generator=g) * torch.exp(3 * torch.randn(m, 1, generator=g))
    _check_quantize(x.to(bf), pitch)


def test_quantize_every_magnitude():
    """Every bf16 value from subnormals to the largest, each block with a maximum of its own."""
    codes = torch.arange(0, 0x7F80, dtype=torch.int32).to(torch.int16)   # 32640 = 255 x 128 non-negative numbers
    x = codes.view(bf).reshape(255, 128)
    _check_quantize(torch.cat([x, -x.flip(1)], dim=1))


def test_quantize_zero_nan_inf():
    x = torch.randn(6, 288, generator=torch.Generator().manual_seed(1)).to(bf)
    x[0] = 0
    x[1, :128] = -0.0
    x[2, 5] = float("nan")
    x[3, 200] = float("inf")
    x[4, 287] = -float("inf")
    _check_quantize(x)


# ----------------------------------------------------------------------------- product
def _data(m, n, k, seed, mats=1):
    r = np.random.default_rng(seed)
    kb, nb = -(-k // 128), -(-n // 128)
    x = fp8.encode(r.standard_normal((m, k)) * 60)
    ws = [fp8.encode(r.standard_normal((n, k)) * 60) for _ in range(mats)]
    xs = (r.uniform(0.5, 2, (kb, m)) / 60).astype(np.float32)
    wss = [(r.uniform(0.25, 4, (nb, kb)) / 60 / np.sqrt(k)).astype(np.float32) for _ in range(mats)]
    return x, xs, ws, wss


def _f8(codes, dev, pitch=0):
    t = torch.zeros(codes.shape[0], codes.shape[1] + pitch, dtype=torch.uint8, device=dev)
    t[:, :codes.shape[1]] = torch.from_numpy(codes).to(dev)
    return t.view(f8)[:, :codes.shape[1]]


def _check(m, n, k, epi, seed=0, pitch=0, in_place=False, out_pitch=0):
    dev = require_gpu()
    swiglu, residual = epi == "swiglu", epi == "residual"
    code = {"bf16": e3.EPI_BF16, "f32": e3.EPI_F32, "residual": e3.EPI_BF16_RESIDUAL, "swiglu": e3.EPI_SWIGLU}[epi]
    x, xs, ws, wss = _data(m, n, k, seed + m + n + k, 2 if swiglu else 1)
    res = torch.randn(m, n, generator=torch.Generator().manual_seed(seed)).to(bf) if residual else None
    out = torch.full((m, n + out_pitch), 7.0, dtype=f32 if epi == "f32" else bf, device=dev)
    if in_place:
        out[:, :n] = res.to(dev)
    st = torch.zeros(1, dtype=i32, device=dev)
    t = lambda a: torch.from_numpy(a).to(dev)
    e3.eagle3_linear_fp8(_f8(x, dev, pitch), t(xs), _f8(ws[0], dev, pitch), t(wss[0]), out[:, :n], epilogue=code,
                         w2=_f8(ws[1], dev, pitch) if swiglu else None, w2_scale=t(wss[1]) if swiglu else None,
                         residual=None if res is None else out[:, :n] if in_place else res.to(dev), dev_status=st)
    torch.cuda.synchronize()
    assert int(st) == 0 and (out[:, n:] == 7).all()
    y, S = fp8.linear(x, xs, ws[0], wss[0])
    tol = (256 + 3 + xs.shape[0]) * U * S
    if swiglu:
        y2, S2 = fp8.linear(x, xs, ws[1], wss[1])
        tol2 = (256 + 3 + xs.shape[0]) * U * S2
        want = moe.silu(y) * y2
        tol = 1.1 * tol * (np.abs(y2) + tol2) + np.abs(moe.silu(y)) * tol2 + 2.0 ** -20 * np.abs(want)
    else:
        want = y
        if residual:
            want = y + _np(res)
            tol = tol + U * np.abs(want)
    if epi != "f32":
        tol = tol + BF16 * (np.abs(want) + tol)
    err = np.abs(_np(out[:, :n]) - want)
    assert (err <= tol + 1e-37).all(), (float((err / (tol + 1e-37)).max()), float(err.max()))


EPIS = ["bf16", "f32", "residual", "swiglu"]


@pytest.mark.parametrize("epi", EPIS)
@pytest.mark.parametrize("m,n,k", [
    (1, 64, 128), (1, 1, 16), (3, 130, 144), (16, 256, 512), (17, 1000, 1024), (33, 96, 2064), (64, 640, 4096),
    (65, 100, 256), (100, 300, 400), (128, 512, 768), (8, 6144, 4096), (24, 19601, 256), (28, 19601, 256)])
def test_fp8_few_rows(m, n, k, epi):
    _check(m, n, k, epi)


@pytest.mark.parametrize("epi", EPIS)
@pytest.mark.parametrize("m,n,k", [
    (129, 64, 128), (130, 1, 16), (200, 130, 144), (256, 512, 256), (300, 777, 1040), (640, 1000, 512),
    (1000, 2560, 384), (513, 600, 4096)])
def test_fp8_many_rows(m, n, k, epi):
    _check(m, n, k, epi)


@pytest.mark.parametrize("epi", EPIS)
@pytest.mark.parametrize("m,n,k", [(70, 130, 4112), (129, 1, 2560), (200, 521, 8192), (100, 2600, 3088),
                                   (1100, 1001, 6160), (1100, 1161, 6160)])
def test_fp8_k_ranges(m, n, k, epi):
    """Few tiles and a long k: the k-blocks are cut over a cluster, with odd ranges and odd columns (the last two by
    tiles of 256 columns, the others of 128)."""
    _check(m, n, k, epi)
    _check(m, n, k, epi, seed=1, out_pitch=3)


@pytest.mark.parametrize("m", [5, 300])
@pytest.mark.parametrize("epi", EPIS)
def test_fp8_pitched_views(m, epi):
    _check(m, 200, 272, epi, pitch=48, out_pitch=8)
    _check(m, 200, 272, epi, out_pitch=3)      # rows that no 16-byte store fits


@pytest.mark.parametrize("m,n,k", [(5, 264, 256), (300, 264, 256), (200, 264, 4096), (300, 263, 256), (2500, 5000, 128),
                                   (2500, 5001, 128)])
def test_fp8_residual_in_place(m, n, k):
    """Every kernel, and several tiles a CTA."""
    _check(m, n, k, "residual", in_place=True)


@pytest.mark.parametrize("m", [4, 200])
def test_fp8_nan_stays_in_its_row_and_column(m):
    dev = require_gpu()
    x, xs, ws, wss = _data(m, 300, 256, 3)
    x[1, 3] = 0x7F
    ws[0][200, 9] = 0xFF
    xs[1, 2] = np.nan
    out = torch.zeros(m, 300, dtype=bf, device=dev)
    t = lambda a: torch.from_numpy(a).to(dev)
    e3.eagle3_linear_fp8(_f8(x, dev), t(xs), _f8(ws[0], dev), t(wss[0]), out)
    nan = torch.isnan(out).cpu().numpy()
    want = np.zeros((m, 300), bool)
    want[1:3] = True
    want[:, 200] = True
    np.testing.assert_array_equal(nan, want)


@pytest.mark.parametrize("m", [4, 200])
def test_fp8_zero_and_large_scales(m):
    """Scales of zero, subnormal scales and scales far apart."""
    dev = require_gpu()
    n, k = 256, 512
    x, xs, ws, wss = _data(m, n, k, 4)
    xs[:] = np.array([0.0, 1e-39, 1e6, 1.0], np.float32)[:, None]
    wss[0][0] = [1.0, 1.0, 1e-6, 1e-3]
    wss[0][1] = [1e5, 1e6, 1e3, 0.0]
    out = torch.zeros(m, n, device=dev)
    t = lambda a: torch.from_numpy(a).to(dev)
    e3.eagle3_linear_fp8(_f8(x, dev), t(xs), _f8(ws[0], dev), t(wss[0]), out, epilogue=e3.EPI_F32)
    y, S = fp8.linear(x, xs, ws[0], wss[0])
    assert (np.abs(_np(out) - y) <= (256 + 3 + 4) * U * S + 1e-37).all()


def test_quantize_then_product_in_a_graph():
    """The two calls as a projection uses them: eager, captured and replayed on other inputs, and
    bit-identical run to run."""
    dev = require_gpu()
    for m, n, k in ((9, 384, 640), (300, 384, 640)):
        _, _, ws, wss = _data(1, n, k, 5)
        w, wsc = _f8(ws[0], dev), torch.from_numpy(wss[0]).to(dev)
        x, q = torch.empty(m, k, dtype=bf, device=dev), torch.empty(m, k, dtype=f8, device=dev)
        s, out = torch.empty(k // 128, m, device=dev), torch.empty(m, n, dtype=bf, device=dev)

        def step():
            e3.eagle3_quantize_fp8(x, q, s)
            e3.eagle3_linear_fp8(q, s, w, wsc, out)

        side = torch.cuda.Stream()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
            step()
        for seed in (1, 2):
            x.copy_(torch.randn(m, k, generator=torch.Generator().manual_seed(seed)).to(bf))
            step()
            torch.cuda.synchronize()
            eager = out.clone()
            codes, scale = fp8.quantize(_np(x).astype(np.float32))
            y, S = fp8.linear(codes, scale, ws[0], wss[0])
            tol = (256 + 3 + k // 128) * U * S
            assert (np.abs(_np(eager) - y) <= tol + BF16 * (np.abs(y) + tol) + 1e-37).all()
            out.zero_()
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, eager)


@pytest.mark.parametrize("m,k,out_pitch", [(17, 128, 0), (200, 128, 0), (200, 128, 1), (100, 4096, 0)])
def test_fp8_extreme_gates(m, k, out_pitch):
    """Gates from -1e18 to 1e18 in every kernel: x[r] = (1, 1, 0, ...) with the scale a, unit weights: both sums
    are a.  Tolerance as in the bf16 tests."""
    dev = require_gpu()
    n, kb = 64, k // 128
    values = [0.0, -0.0, 1.0, -1.0, -20.0, -60.0, -80.0, -87.0, -87.5, -88.0, -89.0, -100.0, 88.0, 100.0, 1e18, -1e18]
    a = np.array([values[i % len(values)] for i in range(m)], np.float32)
    x = np.zeros((m, k), np.uint8)
    wg, wu = np.zeros((n, k), np.uint8), np.zeros((n, k), np.uint8)
    one = fp8.encode(np.ones((1, 1)))[0, 0]
    x[:, k - 2:] = one
    wg[:, k - 2] = wu[:, k - 1] = one
    t = lambda v: torch.from_numpy(v).to(dev)
    xs, ws = np.repeat(a[None], kb, 0), np.ones((1, kb), np.float32)
    out = torch.empty(m, n + out_pitch, dtype=bf, device=dev)[:, :n]
    e3.eagle3_linear_fp8(_f8(x, dev), t(xs), _f8(wg, dev), t(ws), out, epilogue=e3.EPI_SWIGLU, w2=_f8(wu, dev),
                         w2_scale=t(ws))
    a = a.astype(np.float64)
    want = moe.silu(a) * a
    tol = (BF16 + 2 * U * (8 + 1.2 * np.abs(np.clip(a, -100, 100)))) * np.abs(want)
    tol = tol + np.where(a < -87, 2.0 ** -119, 0) * np.abs(a) + 2.0 ** -133
    assert (np.abs(_np(out) - want[:, None]) <= tol[:, None]).all()


@pytest.mark.parametrize("m,n,k", [(20, 200, 256), (200, 200, 256), (200, 200, 4096)])
def test_fp8_offsets_past_32_bits(m, n, k):
    """Rows so far apart that the last ones start past 2^31 elements from the first."""
    dev = require_gpu()
    pitch = (2 ** 31 // (m - 1) // 16 + 2) * 16
    x, xs, ws, wss = _data(m, n, k, 12)
    t = lambda v: torch.from_numpy(v).to(dev)
    xd = torch.empty(m, pitch, dtype=torch.uint8, device=dev)[:, :k]
    xd.copy_(t(x))
    out = torch.empty(m, pitch, dtype=bf, device=dev)[:, :n]
    e3.eagle3_linear_fp8(xd.view(f8), t(xs), _f8(ws[0], dev), t(wss[0]), out)
    y, S = fp8.linear(x, xs, ws[0], wss[0])
    tol = (256 + 3 + xs.shape[0]) * U * S
    assert (np.abs(_np(out) - y) <= tol + BF16 * (np.abs(y) + tol) + 1e-37).all()
    b = torch.empty(m, pitch, dtype=bf, device=dev)[:, :k]
    b.copy_(torch.randn(m, k, generator=torch.Generator().manual_seed(13)))
    scale = torch.empty(-(-k // 128), m, device=dev)
    e3.eagle3_quantize_fp8(b, xd.view(f8), scale)
    codes, want = fp8.quantize(b.float().cpu().numpy())
    np.testing.assert_array_equal(scale.cpu().numpy(), want)
    np.testing.assert_array_equal(xd.cpu().numpy(), codes)


def test_fp8_on_two_streams_at_once():
    """The kernels with and without clusters, side by side."""
    dev = require_gpu()
    t = lambda v: torch.from_numpy(v).to(dev)
    sets = []
    for m, n, k in ((20, 300, 1024), (200, 600, 4096), (700, 1300, 512), (64, 256, 4096)):
        x, xs, ws, wss = _data(m, n, k, 14)
        sets.append([_f8(x, dev), t(xs), _f8(ws[0], dev), t(wss[0]), torch.empty(m, n, dtype=bf, device=dev)])
    run = lambda order: [e3.eagle3_linear_fp8(*sets[i]) for i in order]
    run(range(4))
    torch.cuda.synchronize()
    want = [s[4].clone() for s in sets]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for s in sets:
            s[4].zero_()
        torch.cuda.synchronize()
        for order, stream in zip(((0, 1), (2, 3)), streams):
            with torch.cuda.stream(stream):
                for _ in range(4):
                    run(order)
        torch.cuda.synchronize()
        for s, w in zip(sets, want):
            assert torch.equal(s[4], w)
