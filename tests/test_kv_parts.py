"""Parts that a caller of eagle3_verify_attn_fp8 asks for: at most 512, by both kernels, in a workspace that stays within bounds
(no GPU needed)."""
import ctypes

import pytest

from tests._util import built_lib
from tests.test_kv_abi import _attn

LONG = dict(batch=64, n_nodes=60, n_heads=32, n_kv_heads=8, max_prefix_len=1 << 20, max_blocks=1 << 14, n_pages=1 << 20)


@pytest.mark.parametrize("kernel", [1, 2])
@pytest.mark.parametrize("kw", [{}, LONG, dict(LONG, batch=1), dict(LONG, n_kv_heads=1, n_heads=4)])
def test_more_than_512_parts_are_512(kernel, kw):
    size = lambda splits: built_lib().eagle3_test_verify_attn_fp8_workspace_size(
        ctypes.byref(_attn(**{**dict(n_nodes=60), **kw}, num_splits=splits)), kernel)
    assert 0 < size(512) == size(513) == size(100000) == size(2 ** 31 - 1)


@pytest.mark.parametrize("kw", [LONG, dict(LONG, batch=1), dict(LONG, batch=4096, n_nodes=5), dict(LONG, n_heads=2048)])
@pytest.mark.parametrize("splits", [1, 30, 512])
def test_128_rows_at_a_time_take_a_bounded_workspace(kw, splits):
    """Eight waves of CTAs (152 SMs), each with two units' partial results of 128 rows."""
    size = built_lib().eagle3_test_verify_attn_fp8_workspace_size(ctypes.byref(_attn(**{**kw, "num_splits": splits})), 2)
    groups = -(-kw["n_nodes"] * kw["n_heads"] // kw["n_kv_heads"] // 128)
    ctas = max(8 * 152, groups)
    assert 0 < size <= ctas * 2 * 128 * 130 * 4 + 8 * ctas * 2 + 8 * (kw["batch"] + 3) + 5 * 256
