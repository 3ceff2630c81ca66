"""Refusals of the 8-bit cache's binding that the C calls cannot make (no GPU needed)."""
import pytest
import torch

import eagle_tree_speculative_spec_gb300 as e3

z = torch.zeros


@pytest.mark.parametrize("table", [z(32, 2, dtype=torch.int64), z(1, 32, dtype=torch.int64), z((), dtype=torch.int64)])
def test_append_refuses_a_table_that_is_none(table):
    """A rope table is one row of turns, as eagle3_rope takes it; of another shape its first dim is not a count of pairs."""
    k, i32 = z(6, 2, 64, dtype=torch.bfloat16), torch.int32
    pool = z(192, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="rotary_dim / 2"):
        e3.eagle3_append_kv(k, k, z(2, dtype=i32), z(2, dtype=i32), z(2, 4, dtype=i32), pool, pool, max_new=3, block_size=64,
                            rope_table=table)
