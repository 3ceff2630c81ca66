"""Mixture-of-experts feed-forward: routing, products by expert, weighted sum.

The layer stands where "EAGLE-3: Engineering Implementation of LLM Inference Acceleration",
appendix C has one SwiGLU: with experts e = 1..E, row x takes the k experts of the largest router
logits z_e and
    y = residual + sum over them of weight_e * W_down,e (silu(W_gate,e x) * (W_up,e x)).

Row-at-a-time fp64; ids, offsets and slots are exact integers.

Pinned by: with one expert, or with all experts taken under un-normalised softmax weights and equal
weights matrices, the layer equals the dense SwiGLU (tests/test_oracle_moe_fp8.py); a brute-force
sort of (logit, expert) pairs.
"""
import math

import numpy as np


def route(logits, k, sigmoid=False, renormalize=True, scale=1.0, num_rows=None):
    """(ids [T, k], weights [T, k] fp64, offsets [E + 1], sorted_rows [T * k], slots [T, k])."""
    z = np.asarray(logits, dtype=np.float64)
    T, E = z.shape
    limit = T if num_rows is None else min(max(int(num_rows), 0), T)
    ids = np.full((T, k), -1, dtype=np.int64)
    weights = np.zeros((T, k))
    for t in range(limit):
        usable = [e for e in range(E) if math.isfinite(z[t, e])]
        usable.sort(key=lambda e: (-z[t, e], e))
        take = usable[:k]
        if not take:
            continue
        if sigmoid:
            score = [1.0 / (1.0 + math.exp(-z[t, e])) if z[t, e] > -700 else 0.0 for e in take]
            total = 1.0
        else:
            m = z[t, take[0]]
            score = [math.exp(z[t, e] - m) for e in take]
            total = sum(math.exp(z[t, e] - m) for e in usable)
        if renormalize:
            total = sum(score)
        for j, e in enumerate(take):
            ids[t, j] = e
            weights[t, j] = score[j] / total * scale if total > 0 else 0.0
    offsets = np.zeros(E + 1, dtype=np.int64)
    sorted_rows = np.full(T * k, -1, dtype=np.int64)
    slots = np.full((T, k), -1, dtype=np.int64)
    slot = 0
    for e in range(E):
        for t, j in zip(*np.nonzero(ids == e)):
            sorted_rows[slot] = t
            slots[t, j] = slot
            slot += 1
        offsets[e + 1] = slot
    return ids, weights, offsets, sorted_rows, slots


def silu(x):
    return x / (1.0 + np.exp(-np.clip(x, -700, None)))


def grouped_linear(x, w, offsets, row_ids=None, w2=None):
    """(out [offsets[E], n] fp64, bound [same], gate, up): out[s] = x[r(s)] W_e^T, or SwiGLU with w2;
    bound = sum |x| |w| of the product (the larger of the two products for SwiGLU)."""
    x, w = np.asarray(x, dtype=np.float64), np.asarray(w, dtype=np.float64)
    m, n = int(offsets[-1]), w.shape[1]
    gate, up = np.zeros((m, n)), np.zeros((m, n))
    bound = np.zeros((m, n))
    for e in range(w.shape[0]):
        a, b = int(offsets[e]), int(offsets[e + 1])
        if a == b:
            continue
        rows = x[a:b] if row_ids is None else x[np.asarray(row_ids[a:b])]
        gate[a:b] = rows @ w[e].T
        bound[a:b] = np.abs(rows) @ np.abs(w[e]).T
        if w2 is not None:
            v = np.asarray(w2[e], dtype=np.float64)
            up[a:b] = rows @ v.T
            bound[a:b] = np.maximum(bound[a:b], np.abs(rows) @ np.abs(v).T)
    return (gate if w2 is None else silu(gate) * up), bound, gate, up


def combine(y, slots, weights, residual=None):
    """(out [T, d] fp64, bound): the weighted sum over the slots >= 0 plus the residual."""
    y, weights = np.asarray(y, dtype=np.float64), np.asarray(weights, dtype=np.float64)
    T, k = slots.shape
    out = np.zeros((T, y.shape[1])) if residual is None else np.array(residual, dtype=np.float64)
    bound = np.abs(out)
    for t in range(T):
        for j in range(k):
            if slots[t, j] >= 0:
                v = weights[t, j] * y[slots[t, j]]
                out[t] += v
                bound[t] += np.abs(v)
    return out, bound
