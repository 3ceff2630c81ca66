"""The parts that eagle3_verify_attn_fp8 cuts a prefix into, and their joins, on the GPU, each kernel by its name.

Where a single key has all the weight, the other keys' scores lie some 181 below its own (e^-181 is 0 in fp32), so the output
is that key's value, which bf16 holds: exact but for the 2^x unit and the roundings of a score, below bf16's half step of 2^-8.
Elsewhere the tolerances are those of tests/test_gpu_kv.py.
"""
import ctypes

import numpy as np
import pytest
import torch

from eagle_tree_speculative_spec_gb300 import _lib
from oracle import fp8, kv
from tests._util import require_gpu
from tests.test_gpu_kv import BF16, U, _attn_inputs, _expected, _ints, _np

pytestmark = pytest.mark.gpu

ROWS, WIDE = 1, 2
NAME = {ROWS: "16 rows", WIDE: "128 rows"}
bf, i32, u8, f8 = torch.bfloat16, torch.int32, torch.uint8, torch.float8_e4m3fn


def _run(kernel, pool, lens, q, tk, tv, par, dev, **kw):
    (kc, vc), (ks, vs), table = pool.device()
    out = torch.full(q.shape, 7.0, dtype=bf, device=dev)
    lse = torch.full(q.shape[:3], 7.0, device=dev)
    st = torch.zeros(1, dtype=i32, device=dev)
    t = lambda x: None if x is None else (x if isinstance(x, torch.Tensor) else torch.from_numpy(x)).to(dev)
    _lib.eagle3_test_verify_attn_fp8(q.to(dev), kc, vc, ks, vs, table, _ints(lens, dev), out, kernel=kernel,
                                     max_prefix_len=max(lens), tree_k=t(tk), tree_v=t(tv), parents=t(par), lse=lse,
                                     dev_status=st, **kw)
    torch.cuda.synchronize()
    assert int(st) == 0
    return out, lse


@pytest.mark.parametrize("kernel", [ROWS, WIDE], ids=NAME.get)
@pytest.mark.parametrize("N,splits", [(60, 0), (60, 1), (20, 3), (20, 20)])
@pytest.mark.parametrize("tree", [False, True])
def test_a_nan_scale_of_values_leaves_the_logarithms(kernel, N, splits, tree):
    """The sum of exp has no values in it: V's scale byte 255 makes the outputs NaN, and lse stays what the keys make it."""
    dev = require_gpu()
    lens = [700, 90]
    pool, q, tk, tv, par = _attn_inputs(dev, lens, N, 8, 2, 64, 33, tree)
    pool.scale[1].numpy()[pool.table[0, 3], 1, 0] = 255
    pool.scale[1].numpy()[pool.table[1, 1], 0, 0] = 255     # a group that the sequence ends in
    out, lse = _run(kernel, pool, lens, q, tk, tv, par, dev, num_splits=splits)
    _, want, _, tol = _expected(pool, lens, q, tk, tv, par)
    nan = np.zeros(out.shape, bool)
    nan[0, :, 4:] = nan[1, :, :4] = True
    np.testing.assert_array_equal(np.isnan(_np(out)), nan)
    assert (np.abs(_np(lse) - want) <= tol).all()


# (kernel, sequences, nodes, parts): joins of a CTA's warps, within clusters, by a warp or a CTA a row; of ranges of CTAs
JOINS = [(ROWS, 1, 1, 1), (ROWS, 1, 5, 1), (ROWS, 1, 1, 3), (ROWS, 1, 1, 8), (ROWS, 1, 5, 4), (ROWS, 40, 1, 4), (ROWS, 12, 40, 4),
         (ROWS, 2, 1, 20), (ROWS, 2, 5, 20), (WIDE, 1, 60, 1), (WIDE, 1, 60, 3), (WIDE, 2, 60, 20), (WIDE, 1, 20, 5), (WIDE, 3, 60, 0)]
JOIN_IDS = [f"{NAME[k]}, {b} x {n} nodes, {s} parts" for k, b, n, s in JOINS]


@pytest.mark.parametrize("what", ["nothing", "code", "scale", "tree nan", "tree inf"])
@pytest.mark.parametrize("kernel,B,N,splits", JOINS, ids=JOIN_IDS)
def test_values_that_are_not_finite_far_below_the_maximum(kernel, B, N, splits, what):
    """A NaN code, a NaN scale or a tree's value that is not finite makes the queries that see it so, in whatever part of
    the prefix it lies and however little weight it has; no other query, and not the logarithm of the sum."""
    dev = require_gpu()
    Hq, Hkv, size, L, at = 8, 2, 64, 1500, 1400
    lens = [L] * B
    pool, q, tk, tv, par = _attn_inputs(dev, lens, N, Hq, Hkv, size, 31, True)
    q.zero_()
    q[..., 0] = 64
    tk.zero_()
    tk[..., 0] = -16
    k = pool.codes[0].numpy()
    k[:] = 0
    k[..., 0] = fp8.encode(np.array(-16.0))
    pool.scale[0].numpy()[:] = 127
    for b in range(B):
        k[pool.table[b, 0], :, 0, 0] = fp8.encode(np.array(16.0))
    first = np.stack([kv.read(pool.codes[1].numpy(), pool.scale[1].numpy(), pool.table[b].tolist(), 1, pool.pages)[:, 0]
                      for b in range(B)])                    # [B, Hkv, D]: the value of the key that has the weight
    want = np.repeat(first, Hq // Hkv, 1)[:, None].repeat(N, 1)
    node = N - 1 if N > 32 else N // 2
    sees = np.array([node in kv.path(par[0], i) for i in range(N)])
    if what == "code":
        pool.codes[1].numpy()[pool.table[0, at // size], 1, at % size, 5] = 0xFF
        want[0, :, 4:, 5] = np.nan
    elif what == "scale":
        pool.scale[1].numpy()[pool.table[0, at // size], 0, 0] = 255
        want[0, :, :4] = np.nan
    elif what != "nothing":
        tv[0, node, 1, 7] = float(what.split()[1])
        want[0, sees, 4:, 7] = float(what.split()[1])
    out, lse = _run(kernel, pool, lens, q, tk, tv, par, dev, num_splits=splits)
    got = _np(out)
    np.testing.assert_array_equal(np.isnan(got), np.isnan(want))
    inf = np.isinf(want)
    np.testing.assert_array_equal(got[inf], want[inf])
    ok = np.isfinite(want)
    assert (np.abs(got[ok] - want[ok]) <= BF16 * np.abs(want[ok])).all()
    score = 64 * 16 / 128 ** 0.5
    # the sum of exp is 1; the score: 6 roundings and 2^x's unit, 128 products of which all but one are zeros
    assert (np.abs(_np(lse) - score) <= (6 + 8) * U * score + 2.0 ** -21).all()


@pytest.mark.parametrize("kernel", [ROWS, WIDE], ids=NAME.get)
def test_more_than_512_parts_give_the_same_bits(kernel):
    dev = require_gpu()
    lens = [20000, 300]
    pool, q, tk, tv, par = _attn_inputs(dev, lens, 20, 8, 1, 64, 37, True)
    outs = [_run(kernel, pool, lens, q, tk, tv, par, dev, num_splits=s) for s in (512, 513, 2 ** 31 - 1)]
    for out, lse in outs[1:]:
        assert torch.equal(out, outs[0][0]) and torch.equal(lse, outs[0][1])
    want, _, tol, _ = _expected(pool, lens, q, tk, tv, par)
    assert (np.abs(_np(outs[0][0]) - want) <= tol).all()


@pytest.mark.parametrize("B,N,splits", [(1, 1, 2), (1, 1, 8), (2, 3, 2), (1, 5, 4), (40, 1, 3)])
def test_parts_asked_for_need_their_workspace(B, N, splits):
    """However they are joined: a size that depends on the sizes alone, and a refusal without it."""
    dev = require_gpu()
    pool, q, *_ = _attn_inputs(dev, [500] * B, N, 8, 2, 64, 36, False)
    (kc, vc), (ks, vs), table = pool.device()
    out, q = torch.full(q.shape, 7.0, dtype=bf, device=dev), q.to(dev)
    a = _lib.verify_attn_fp8_args(q, kc, vc, ks, vs, table, _ints([500] * B, dev), out, max_prefix_len=500, num_splits=splits)
    L = _lib.lib()
    need = L.eagle3_verify_attn_fp8_workspace_size(ctypes.byref(a))
    assert need >= splits * B * N * 8 * 130 * 4
    stream = torch.cuda.current_stream().cuda_stream
    assert L.eagle3_verify_attn_fp8(ctypes.byref(a), None, 0, stream) == 6
    ws = torch.empty(need, dtype=u8, device=dev)
    assert L.eagle3_verify_attn_fp8(ctypes.byref(a), ws.data_ptr(), need - 1, stream) == 6
    torch.cuda.synchronize()
    assert (out == 7).all()
    assert L.eagle3_verify_attn_fp8(ctypes.byref(a), ws.data_ptr(), need, stream) == 0
    torch.cuda.synchronize()
    assert not (out == 7).all()


@pytest.mark.parametrize("lens,N,Hq,splits", [([3000, 40], 20, 8, 47), ([3000, 0], 17, 16, 33), ([1500, 600], 33, 4, 12),
                                              ([9000], 20, 2, 2000), ([1500, 9] * 4, 30, 4, 8), ([1000], 64, 8, 5)])
@pytest.mark.parametrize("tree", [False, True])
def test_many_parts_of_128_rows(lens, N, Hq, splits, tree):
    dev = require_gpu()
    pool, q, tk, tv, par = _attn_inputs(dev, lens, N, Hq, 2 if Hq > 2 else 1, 64, 35, tree)
    out, lse = _run(WIDE, pool, lens, q, tk, tv, par, dev, num_splits=splits)
    want, want_lse, tol, lse_tol = _expected(pool, lens, q, tk, tv, par)
    assert (np.abs(_np(out) - want) <= tol).all()
    got, empty = _np(lse), np.isinf(want_lse)
    assert (got[empty] == -np.inf).all()
    assert (np.abs(got[~empty] - want_lse[~empty]) <= lse_tol[~empty]).all()


@pytest.mark.parametrize("B,splits", [(1, 3), (1, 8), (2, 20), (20, 4)])
def test_nan_in_one_part_of_128_rows(B, splits):
    """A NaN key or value in one of many parts reaches its sequence's rows of that KV head, and no others."""
    dev = require_gpu()
    N, lens = 20, [1500] * B
    pool, q, tk, tv, par = _attn_inputs(dev, lens, N, 8, 2, 64, 13, False)
    pool.codes[0].numpy()[pool.table[0, 11], 0, 9, 3] = 0x7F
    pool.codes[1].numpy()[pool.table[B - 1, 20], 1, 9, 5] = 0xFF
    out, _ = _run(WIDE, pool, lens, q, tk, tv, par, dev, num_splits=splits)
    want = np.zeros(out.shape, bool)
    want[0, :, :4] = True
    want[B - 1, :, 4:, 5] = True
    np.testing.assert_array_equal(torch.isnan(out).cpu().numpy(), want)
