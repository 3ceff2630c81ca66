"""e4m3 values with block scales: quantisation and the scaled matrix product.

e4m3 here is the 8-bit format without infinities: sign, 4 exponent bits with bias 7, 3 fraction bits;
exponent 0 is subnormal (steps of 2^-9), the largest value is 448 (0x7E), 0x7F is NaN.

Pinned by: the known values of the format and torch's own conversions (tests/test_oracle_moe_fp8.py).
"""
import numpy as np

MAX = 448.0
BLOCK = 128


def _table():
    v = np.empty(256)
    for c in range(256):
        e, f = (c >> 3) & 15, c & 7
        mag = f * 2.0 ** -9 if e == 0 else (1 + f / 8) * 2.0 ** (e - 7)
        if c & 0x7F == 0x7F:
            mag = np.nan
        v[c] = -mag if c & 0x80 else mag
    return v


TABLE = _table()


def decode(codes):
    return TABLE[np.asarray(codes, dtype=np.uint8)]


def encode(v):
    """Nearest e4m3 code (ties to the even code), magnitudes above 448 to 448, NaN to NaN."""
    v = np.asarray(v, dtype=np.float64)
    grid = TABLE[:0x7F]                                    # 0 .. 448, increasing; code = index
    mag = np.minimum(np.abs(v), MAX)
    mag = np.where(np.isnan(mag), 0.0, mag)
    hi = np.clip(np.searchsorted(grid, mag), 1, 0x7E)      # grid[hi - 1] < mag <= grid[hi] (or mag = 0)
    lo = hi - 1
    up = (mag - grid[lo] > grid[hi] - mag) | ((mag - grid[lo] == grid[hi] - mag) & (hi % 2 == 0))
    code = np.where(up, hi, lo)
    code = code | np.where(np.signbit(v), 0x80, 0)
    return np.where(np.isnan(v), 0x7F, code).astype(np.uint8)


def quantize(x):
    """x [m, k] (fp32 values): (codes [m, k] uint8, scale [ceil(k / 128), m] fp32).  The scale and the
    quotient are single IEEE fp32 divisions."""
    x = np.asarray(x, dtype=np.float32)
    m, k = x.shape
    kb = -(-k // BLOCK)
    codes = np.zeros((m, k), dtype=np.uint8)
    scale = np.zeros((kb, m), dtype=np.float32)
    for b in range(kb):
        blk = x[:, b * BLOCK:(b + 1) * BLOCK]
        a = np.abs(blk).max(axis=1)
        s = np.where(a > 0, a / np.float32(MAX), np.float32(1)).astype(np.float32)
        s = np.where(np.isfinite(blk).all(axis=1), s, np.float32(np.nan))
        scale[b] = s
        with np.errstate(invalid="ignore"):
            codes[:, b * BLOCK:(b + 1) * BLOCK] = encode((blk / s[:, None]).astype(np.float32))
    return codes, scale


def linear(x_codes, x_scale, w_codes, w_scale):
    """(y [m, n] fp64, bound): the block-scaled product and the sum of its terms' magnitudes."""
    x, w = decode(x_codes), decode(w_codes)
    m, k = x.shape
    n = w.shape[0]
    y, bound = np.zeros((m, n)), np.zeros((m, n))
    for b in range(-(-k // BLOCK)):
        xs = np.asarray(x_scale[b], dtype=np.float64)[:, None]
        ws = np.repeat(np.asarray(w_scale[:, b], dtype=np.float64), BLOCK)[:n][None, :]
        xb, wb = x[:, b * BLOCK:(b + 1) * BLOCK], w[:, b * BLOCK:(b + 1) * BLOCK]
        y += xs * ws * (xb @ wb.T)
        bound += np.abs(xs * ws) * (np.abs(xb) @ np.abs(wb).T)
    return y, bound
