"""eagle3_append_kv at its edges, on the GPU.  Everything is compared bit by bit."""
import pytest
import torch

import eagle_tree_speculative_spec_gb300 as e3
from tests._util import require_gpu
from tests.test_gpu_kv import Pool, _ints, _table

pytestmark = pytest.mark.gpu

CAPACITY, BAD_TOKEN = 0x4, 0x2
bf, i32, u8 = torch.bfloat16, torch.int32, torch.uint8


@pytest.mark.parametrize("how", ["start", "padded", "ids"])
@pytest.mark.parametrize("turned", [False, True])
def test_append_of_no_rows(how, turned):
    """Tensors of no rows: nothing happens where no sequence has new tokens, and tokens that it is said to have are missing rows."""
    dev = require_gpu()
    Hkv, D, lens = 2, 64, [70, 0, 3]
    pool = Pool(dev, [n + 8 for n in lens], Hkv, D, 64, 1).fill(lens)
    (kc, vc), (ks, vs), table = pool.device()
    none = torch.empty(0, 2 * Hkv, D, dtype=bf, device=dev)
    kw = dict(start=dict(row_start=_ints([0, 0, 0], dev)), padded={},
              ids=dict(row_ids=_ints([[0, -1, -1]] * 3, dev), rows_per_seq=4))[how]
    if turned:
        kw["rope_table"] = _table(dev, D)[0]
    st = torch.zeros(1, dtype=i32, device=dev)
    for new, want in (([0, 0, 0], 0), ([0, 1, 0], BAD_TOKEN)):
        e3.eagle3_append_kv(none[:, :Hkv], none[:, Hkv:], _ints(lens, dev), _ints(new, dev), table, kc, vc, max_new=3,
                            block_size=64, k_scale=ks, v_scale=vs, dev_status=st, **kw)
        assert int(st) == want
        for got, was in zip((kc, vc), pool.codes):
            assert torch.equal(got.view(u8).cpu(), was)
    big = [torch.full((64, Hkv, D), 9.0, dtype=bf, device=dev) for _ in range(2)]
    st.zero_()
    e3.eagle3_append_kv(none[:, :Hkv], none[:, Hkv:], _ints(lens, dev), _ints([0, 0, 0], dev), table[:, :1].contiguous(), *big,
                        max_new=3, block_size=16, dev_status=st, **kw)
    assert int(st) == CAPACITY   # (the first sequence is longer than its one page)
    assert all((t == 9).all() for t in big)
