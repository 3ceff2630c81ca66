"""Pins of the 8-bit cache's oracle: rotations, scale bytes, appends and attention against other forms (no GPU)."""
import math

import numpy as np
import pytest

from oracle import attention as oatt
from oracle import fp8, kv


def test_half_rotation_is_the_model_rotation():
    r = np.random.default_rng(0)
    x, pos = r.standard_normal((9, 3, 16)), r.integers(0, 5000, 9)
    got = kv.rope(x, pos, kv.frequencies(16, 10000.0))
    # that one takes its angles in fp32: off by up to 5000 * 2^-23
    assert np.abs(got - oatt.rope_apply(x, pos, 10000.0)).max() < 5000 * 2.0 ** -22


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rotation_is_a_complex_product_and_inverts(layout):
    r = np.random.default_rng(1)
    x, pos = r.standard_normal((5, 2, 24)), r.integers(-100, 1 << 20, 5)
    f = kv.frequencies(20, 500000.0, "ramp", 8.0, 1.0, 32.0, 4096)
    y = kv.rope(x, pos, f, layout, amplitude=1.25)
    a, b = kv.pairs(20, layout)
    z = (x[..., a] + 1j * x[..., b]) * 1.25 * np.exp(1j * pos[:, None, None] * f)
    assert np.allclose(y[..., a], z.real, atol=1e-9) and np.allclose(y[..., b], z.imag, atol=1e-9)
    assert (y[..., 20:] == x[..., 20:]).all()
    back = kv.rope(y, pos, f, layout, inverse=True, amplitude=1 / 1.25)
    assert np.allclose(back, x, atol=1e-9)


def test_frequencies():
    f = kv.frequencies(8, 10000.0)
    assert np.allclose(f, [1, 0.1, 0.01, 0.001])
    assert np.allclose(kv.frequencies(8, 10000.0, "linear", 4.0), f / 4)
    # the last pair of a stretched base turns as if the positions were divided by the factor
    assert math.isclose(kv.frequencies(8, 10000.0, "base", 4.0)[-1], f[-1] / 4)
    b = kv.frequencies(128, 500000.0, "bands", 8.0, 1.0, 4.0, 8192)
    plain = kv.frequencies(128, 500000.0)
    wl = 2 * np.pi / plain
    assert (b[wl < 2048] == plain[wl < 2048]).all() and np.allclose(b[wl > 8192], plain[wl > 8192] / 8)
    assert (np.diff(b) < 0).all()
    r = kv.frequencies(128, 500000.0, "ramp", 8.0, 1.0, 32.0, 8192)
    assert r[0] == plain[0] and math.isclose(r[-1], plain[-1] / 8) and (np.diff(r / plain) <= 1e-12).all()


def test_scale_byte():
    for e in (-100, -3, 0, 5, 100):
        top = 448.0 * 2.0 ** e
        assert kv.scale_byte(top) == 127 + e and kv.scale_byte(top * (1 + 2 ** -23)) == 128 + e
    assert kv.scale_byte(0.0) == 1 and kv.scale_byte(1e-45) == 1


def _pool(pages, heads, size, dim):
    return np.zeros((pages, heads, size, dim), np.uint8), np.zeros((pages, heads, size // 64), np.uint8)


def test_append_token_by_token_is_append_at_once_up_to_the_scales_growth():
    r = np.random.default_rng(2)
    rows = r.standard_normal((150, 2, 8)) * np.exp(r.standard_normal((150, 1, 1)))
    table = [2, 0, 3]
    one, s1 = _pool(4, 2, 64, 8)
    many, s2 = _pool(4, 2, 64, 8)
    kv.append(one, s1, table, 0, rows, 4)
    for i in range(150):
        kv.append(many, s2, table, i, rows[i:i + 1], 4)
    assert (s1 == s2).all() and (s1[1] == 0).all()
    a, b = (kv.read(c, s, table, 150, 4) for c, s in ((one, s1), (many, s2)))
    want = rows.transpose(1, 0, 2)
    f = np.concatenate([np.repeat(2.0 ** (s1[p, :, 0].astype(int) - 127)[:, None], 64, 1) for p in table], 1)[:, :150, None]
    half = np.maximum(np.abs(want) * 2.0 ** -4, f * 2.0 ** -10)
    assert (np.abs(a - want) <= half).all()
    # a second rounding can only happen in the subnormals of the scale that grew
    assert (np.abs(b - want) <= half + f * 2.0 ** -10).all()
    assert (one[2, :, :, :] == fp8.encode(rows[:64].transpose(1, 0, 2) / f[:, :64])).all()


def test_append_keeps_other_places_and_marks_non_finite_values():
    codes, scale = _pool(2, 1, 128, 8)
    codes[:] = 0x55
    rows = np.ones((3, 1, 8))
    rows[1, 0, 2], rows[2, 0, 5] = np.inf, np.nan
    kv.append(codes, scale, [1], 70, rows, 2)
    got = codes[1, 0, 70:73]
    assert got[1, 2] == 0x7F and got[2, 5] == 0x7F and scale[1, 0, 1] == kv.scale_byte(1.0) and scale[1, 0, 0] == 0
    assert (codes[0] == 0x55).all() and (codes[1, 0, 73:] == 0x55).all() and (codes[1, 0, :64] == 0x55).all()


def test_attention_is_the_tree_attention():
    r = np.random.default_rng(3)
    N, Hq, Hkv, D, L = 7, 4, 2, 16, 37
    q, tk, tv = r.standard_normal((1, N, Hq, D)), r.standard_normal((1, N, Hkv, D)), r.standard_normal((1, N, Hkv, D))
    k, v = r.standard_normal((1, Hkv, L, D)), r.standard_normal((1, Hkv, L, D))
    par = np.array([[-1, 0, 0, 1, 1, 3, 2]])
    # that one rotates q and the tree keys itself: hand it what it will turn into ours
    pos = np.array([L + len(kv.path(par[0], i)) - 1 for i in range(N)])
    freq = kv.frequencies(D, 10000.0)
    want, lse, rot = oatt.verify_attention(q, tk, tv, k, v, par, np.array([L]), theta=10000.0)
    got, got_lse, _, _ = kv.attention(kv.rope(q[0], pos, freq), k[0], v[0], kv.rope(tk[0], pos, freq), tv[0], par[0])
    assert np.abs(got - want[0]).max() < 1e-4 and np.abs(got_lse - lse[0]).max() < 1e-4


def test_attention_without_keys():
    out, lse, _, _ = kv.attention(np.ones((2, 2, 4)), np.zeros((1, 0, 4)), np.zeros((1, 0, 4)))
    assert (out == 0).all() and (lse == -np.inf).all()
