"""An e4m3 paged KV cache: rotary positions, appends with a power-of-two scale for each 64 places and head, and the
attention that reads it, in 64 bits.

Sources: "EAGLE-3: Engineering Implementation of LLM Inference Acceleration", appendix C (rotate-half RoPE, GQA);
"Speculative Decoding (EAGLE3) in the vLLM Neuron Framework", "EagleProposer: Draft Model Management" (pages);
"Advanced speculative decoding: tree drafts and EAGLE", "Implementation" (a node sees the prefix, its ancestors and
itself).

Pinned by: oracle.attention's rotation and tree attention, complex rotations, and a cache filled token by token against
one filled at once (tests/test_oracle_kv.py).
"""
import math

import numpy as np

from oracle import fp8

GROUP = 64


def frequencies(rotary_dim, theta, scaling="none", factor=1.0, low_turns=1.0, high_turns=4.0, original=8192):
    """Radians a position of every pair."""
    R = rotary_dim
    if scaling == "base":
        theta = theta * factor ** (R / (R - 2))
    f = np.array([theta ** (-2.0 * j / R) for j in range(R // 2)])
    if scaling == "linear":
        return f / factor
    if scaling == "bands":
        out = []
        for w in f:
            wavelength = 2 * math.pi / w
            if wavelength <= original / high_turns:
                out.append(w)
            elif wavelength >= original / low_turns:
                out.append(w / factor)
            else:
                k = (original / wavelength - low_turns) / (high_turns - low_turns)
                out.append(k * w + (1 - k) * w / factor)
        return np.array(out)
    if scaling == "ramp":
        d = lambda t: R * math.log(original / (2 * math.pi * t)) / (2 * math.log(theta))
        lo, hi = max(math.floor(d(high_turns)), 0), min(math.ceil(d(low_turns)), R - 1)
        k = np.clip((np.arange(R // 2) - lo) / max(hi - lo, 0.001), 0, 1)
        return (1 - k) * f + k * f / factor
    return f


def pairs(rotary_dim, layout):
    j = np.arange(rotary_dim // 2)
    return (j, j + rotary_dim // 2) if layout == "half" else (2 * j, 2 * j + 1)


def rope(x, positions, freq, layout="half", inverse=False, amplitude=1.0):
    """x [T, H, D] at positions [T]: the first 2 len(freq) dims of every head turned."""
    y = np.array(x, dtype=np.float64)
    if len(freq) == 0:
        return y
    a, b = pairs(2 * len(freq), layout)
    t = np.asarray(positions, dtype=np.float64)[:, None, None] * freq
    c, s = np.cos(t) * amplitude, np.sin(t) * amplitude * (-1 if inverse else 1)
    xa, xb = y[..., a], y[..., b]
    y[..., a], y[..., b] = xa * c - xb * s, xb * c + xa * s
    return y


def scale_byte(m):
    """The least byte s >= 1 with m <= 448 * 2^(s - 127)."""
    s = 1
    while m > 448.0 * 2.0 ** (s - 127):
        s += 1
    return s


def factor_of(byte):
    return np.nan if byte == 255 else 2.0 ** (int(byte) - 127)


def append(codes, scale, block_table, cache_len, rows, n_pages):
    """One sequence's new rows [n, Hkv, D] (values) at positions cache_len .. into codes [pages, Hkv, size, D] and
    scale [pages, Hkv, size / 64], in place, group by group."""
    size = codes.shape[2]
    n = len(rows)
    p = cache_len
    while p < cache_len + n:
        end = min((p // GROUP + 1) * GROUP, cache_len + n)
        page, place = block_table[p // size], p % size
        g, lo = place // GROUP, place % GROUP
        if 0 <= page < n_pages:
            for h in range(codes.shape[1]):
                new = np.asarray(rows[p - cache_len:end - cache_len, h], dtype=np.float64)
                new = np.where(np.isfinite(new), new, np.nan)
                mags = np.abs(new[np.isfinite(new)])
                s = scale_byte(mags.max() if mags.size else 0.0)
                old = int(scale[page, h, g])
                if lo > 0:
                    s = max(s, old)
                    if s > old:
                        block = codes[page, h, g * GROUP:g * GROUP + lo]
                        again = fp8.encode(fp8.decode(block) * 2.0 ** (old - s))
                        codes[page, h, g * GROUP:g * GROUP + lo] = np.where(np.isnan(fp8.decode(block)), 0x7F, again)
                scale[page, h, g] = s
                codes[page, h, place:place + end - p] = fp8.encode(new / factor_of(s))
        p = end


def read(codes, scale, block_table, length, n_pages):
    """[Hkv, length, D]: what the first positions of a sequence stand for (0 where a page is not in the pool)."""
    size = codes.shape[2]
    out = np.zeros((codes.shape[1], length, codes.shape[3]))
    for p in range(0, length, GROUP):
        page, place = block_table[p // size], p % size
        if 0 <= page < n_pages:
            n = min(GROUP, length - p)
            f = np.array([factor_of(b) for b in scale[page, :, place // GROUP]])
            out[:, p:p + n] = fp8.decode(codes[page, :, place:place + n]) * f[:, None, None]
    return out


def path(parents, i):
    """Nodes that node i sees (up to a parent that is none)."""
    seen = [i]
    while i > 0 and 0 <= parents[i] < i:
        i = parents[i]
        seen.append(i)
    return seen


def attention(q, k, v, tree_k=None, tree_v=None, parents=None, sm_scale=0.0):
    """One sequence: q [N, Hq, D] over k, v [Hkv, L, D] and the tree [N, Hkv, D].  Returns out [N, Hq, D], lse [N, Hq],
    the weighted mean magnitude of the values [N, Hq, D] and the largest sum of |q k| sm_scale over the keys [N, Hq]."""
    N, Hq, D = q.shape
    rep = Hq // k.shape[0]
    sc = sm_scale if sm_scale else 1.0 / math.sqrt(D)
    out, mag = np.zeros((N, Hq, D)), np.zeros((N, Hq, D))
    lse, dot = np.full((N, Hq), -np.inf), np.zeros((N, Hq))
    for i in range(N):
        for h in range(Hq):
            g = h // rep
            ks, vs = k[g], v[g]
            if tree_k is not None:
                own = path(parents, i)
                ks, vs = np.concatenate([ks, tree_k[own, g]]), np.concatenate([vs, tree_v[own, g]])
            if len(ks) == 0:
                continue
            z = ks @ q[i, h] * sc
            m = z.max()
            e = np.exp(z - m)
            out[i, h] = e @ vs / e.sum()
            mag[i, h] = e @ np.abs(vs) / e.sum()
            lse[i, h] = m + math.log(e.sum())
            dot[i, h] = (np.abs(ks) @ np.abs(q[i, h])).max() * sc
    return out, lse, mag, dot
