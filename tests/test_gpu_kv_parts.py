"""The parts that eagle3_verify_attn_fp8 cuts a prefix into, and their joins, on the GPU, each kernel by its name.

The tolerances are those of tests/test_gpu_kv.py.
"""
import numpy as np
import pytest
import torch

from eagle_tree_speculative_spec_gb300 import _lib
from tests._util import require_gpu
from tests.test_gpu_kv import _attn_inputs, _expected, _ints, _np

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
