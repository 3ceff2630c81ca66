"""Pins of the oracle's mixture-of-experts and 8-bit functions (CPU only)."""
from fractions import Fraction

import numpy as np
import pytest
import torch

from oracle import fp8, moe


# ----------------------------------------------------------------------------- e4m3
def test_e4m3_known_values():
    assert fp8.decode([0x00, 0x01, 0x07, 0x08, 0x38, 0x7E, 0xB8]).tolist() == [
        0.0, 2.0 ** -9, 7 * 2.0 ** -9, 2.0 ** -6, 1.0, 448.0, -1.0]
    assert np.isnan(fp8.decode([0x7F, 0xFF])).all()


def test_e4m3_matches_torch():
    codes = torch.arange(256, dtype=torch.uint8)
    ref = codes.view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(fp8.decode(codes.numpy()), ref)
    r = np.random.default_rng(1)
    v = np.concatenate([r.standard_normal(4000) * 10.0 ** r.uniform(-4, 2.6, 4000), fp8.TABLE[:0x7F],
                        (fp8.TABLE[:0x7E] + fp8.TABLE[1:0x7F]) / 2]).astype(np.float32)   # values and ties
    v = np.clip(np.concatenate([v, -v]), -448, 448)
    want = torch.from_numpy(v).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    np.testing.assert_array_equal(fp8.encode(v), want)
    assert fp8.encode([1e9, -np.inf, np.nan]).tolist() == [0x7E, 0xFE, 0x7F]


def test_quantize_blocks():
    x = np.zeros((3, 160), dtype=np.float32)
    x[0, 5] = -896.0
    x[1, 130] = 3.5
    x[2, 7] = np.inf
    q, s = fp8.quantize(x)
    assert s.shape == (2, 3)
    assert s[0, 0] == 2.0 and s[1, 0] == 1.0 and s[0, 1] == 1.0 and s[1, 1] == np.float32(3.5 / 448)
    assert fp8.decode(q)[0, 5] == -448.0 and fp8.decode(q)[1, 130] == 448.0
    assert np.isnan(s[0, 2]) and (q[2, :128] == 0x7F).all() and (q[2, 128:] == 0).all()


def test_scaled_product_is_the_product_of_the_dequantised():
    r = np.random.default_rng(2)
    m, n, k = 5, 140, 300
    x, w = fp8.encode(r.standard_normal((m, k))), fp8.encode(r.standard_normal((n, k)))
    xs, ws = r.uniform(0.5, 2, (3, m)), r.uniform(0.5, 2, (2, 3))
    xd = fp8.decode(x) * np.repeat(xs, 128, axis=0)[:k].T
    wd = fp8.decode(w) * np.repeat(np.repeat(ws, 128, axis=0)[:n], 128, axis=1)[:, :k]
    y, bound = fp8.linear(x, xs, w, ws)
    np.testing.assert_allclose(y, xd @ wd.T, rtol=1e-12, atol=1e-12)
    np.testing.assert_allclose(bound, np.abs(xd) @ np.abs(wd).T, rtol=1e-12)


# ----------------------------------------------------------------------------- experts
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("renormalize", [False, True])
def test_route_order_and_weights(sigmoid, renormalize):
    z = np.array([[0.0, 2.0, 2.0, -1.0], [1.0, -np.inf, np.nan, np.inf], [-np.inf] * 4, [3.0, 1.0, 2.0, 0.0]])
    ids, w, off, rows, slots = moe.route(z, 2, sigmoid, renormalize, 2.0, num_rows=3)
    assert ids.tolist() == [[1, 2], [0, -1], [-1, -1], [-1, -1]]   # the tie goes to the lower expert
    assert off.tolist() == [0, 1, 2, 3, 3] and rows.tolist() == [1, 0, 0, -1, -1, -1, -1, -1]
    assert slots.tolist() == [[1, 2], [0, -1], [-1, -1], [-1, -1]]
    score = 1 / (1 + np.exp(-2.0)) if sigmoid else np.exp(2.0) / np.exp([0.0, 2.0, 2.0, -1.0]).sum()
    np.testing.assert_allclose(w[0], [1.0, 1.0] if renormalize else [2 * score] * 2)
    assert w[1, 1] == 0 and (w[2:] == 0).all()


def test_layer_with_equal_experts_is_the_dense_layer():
    r = np.random.default_rng(3)
    T, E, k, d, F = 6, 4, 4, 10, 7
    x = r.standard_normal((T, d))
    wg, wu, wd = r.standard_normal((F, d)), r.standard_normal((F, d)), r.standard_normal((d, F))
    dense = x + (moe.silu(x @ wg.T) * (x @ wu.T)) @ wd.T
    rep = lambda w: np.stack([w] * E)
    for kk, renorm in ((k, False), (2, True)):   # the weights sum to one either way
        ids, w, off, rows, slots = moe.route(r.standard_normal((T, E)), kk, renormalize=renorm)
        h = moe.grouped_linear(x, rep(wg), off, rows, rep(wu))[0]
        y = moe.grouped_linear(h, rep(wd), off)[0]
        np.testing.assert_allclose(moe.combine(y, slots, w, x)[0], dense, rtol=1e-12, atol=1e-12)


# ----------------------------------------------------------------------------- quotients by correction
def _rn(f):
    """A Fraction to the nearest number of 24 significant bits, ties to even."""
    if f == 0:
        return f
    sign, f = (-1 if f < 0 else 1), abs(f)
    e = f.numerator.bit_length() - f.denominator.bit_length()
    e -= Fraction(2) ** e > f
    u = Fraction(2) ** (e - 23)
    n, rest = divmod(f / u, 1)
    n = int(n) + (rest > Fraction(1, 2) or (rest == Fraction(1, 2) and int(n) % 2 == 1))
    return sign * n * u


def test_corrected_quotients_are_correctly_rounded():
    """What the quantisation kernel relies on: for every significand of a block's maximum and of a value,
    scale, reciprocal and quotient by one correction step are the correctly rounded ones."""
    y448 = _rn(Fraction(1, 448))
    assert float(y448).hex() == "0x1.24924a0000000p-9"
    for top in range(128, 256):
        a = Fraction(top)
        q0 = _rn(a * y448)
        s = _rn(a / 448)
        assert _rn(q0 + _rn(a - q0 * 448) * y448) == s
        y = _rn(1 / s)
        e = y.numerator.bit_length() - y.denominator.bit_length()
        step = Fraction(2) ** (e - (Fraction(2) ** e > y) - 23)
        for d in range(-3, 4):
            y0 = y + d * step
            assert _rn(y0 + y0 * _rn(1 - s * y0)) == y
        for x in range(128, 256):
            q0 = _rn(x * y)
            assert _rn(q0 + _rn(x - q0 * s) * y) == _rn(x / s)
