"""eagle3_append_kv at its edges, on the GPU.  Everything is compared bit by bit."""
import numpy as np
import pytest
import torch

import eagle_tree_speculative_spec_gb300 as e3
from oracle import kv
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


@pytest.mark.parametrize("size", [1, 16, 17, 64, 100])
@pytest.mark.parametrize("many", [False, True])
def test_append_bf16_leaves_out_what_is_wrong(many, size):
    """Counts, lengths, pages and rows out of range: with bf16 pages the tokens of the page that is not there, and no others."""
    dev = require_gpu()
    Hkv, D, W, reach = 2, 64, 70 if many else 4, 140
    lens = [0, 10, -1, reach - 1, 5, 60, 3, 62]
    new = [W, W + 1, 1, 2 + size, -1, W, 0, 4]
    B, columns = len(lens), -(-reach // size)
    pages = B * columns
    g = torch.Generator().manual_seed(size)
    table = torch.randperm(pages, generator=g).reshape(B, columns).numpy().astype(np.int32)
    gone = [(5, 62 // size, pages), (7, 64 // size, -3)]     # pages that are not in the pool, inside a group where they are small
    for b, c, page in gone:
        table[b, c] = page
    rows = torch.randn(B * W, 2 * Hkv, D, generator=g).to(bf)
    start = [b * W for b in range(B)]
    start[0] = B * W - 2                                     # runs past the rows: two tokens only
    pools = [torch.full((pages * size, Hkv, D), 9.0, dtype=bf, device=dev) for _ in range(2)]
    st = torch.zeros(1, dtype=i32, device=dev)
    rd = rows.to(dev)
    e3.eagle3_append_kv(rd[:, :Hkv], rd[:, Hkv:], _ints(lens, dev), _ints(new, dev), torch.from_numpy(table).to(dev), *pools,
                        max_new=W, block_size=size, row_start=_ints(start, dev), dev_status=st)
    assert int(st) == (CAPACITY | BAD_TOKEN)
    for t in range(2):
        want = torch.full((pages * size, Hkv, D), 9.0, dtype=bf)
        for b in (0, 5, 7):
            for j in range(new[b]):
                pos, row = lens[b] + j, start[b] + j
                page = table[b, pos // size]
                if row < B * W and 0 <= page < pages:
                    want[page * size + pos % size] = rows[row, t * Hkv:(t + 1) * Hkv]
        assert torch.equal(pools[t].cpu(), want)


@pytest.mark.parametrize("new", [1, 5, 90])
@pytest.mark.parametrize("R", [0, 64, 20])
def test_append_keeps_the_places_that_no_token_goes_to(new, R):
    """Codes of other places keep their bits, older ones of a group whose scale stays among them."""
    dev = require_gpu()
    Hkv, D, size, lens = 2, 64, 128, [40, 0, 127]
    pool = Pool(dev, [n + new for n in lens], Hkv, D, size, new + R).fill(lens, spread=64.0)
    g = torch.Generator().manual_seed(2)
    rows = torch.randn(3 * new, 2 * Hkv, D, generator=g).to(bf).to(dev)     # far below the older ones: no scale grows
    (kc, vc), (ks, vs), table = pool.device()
    st = torch.zeros(1, dtype=i32, device=dev)
    e3.eagle3_append_kv(rows[:, :Hkv], rows[:, Hkv:], _ints(lens, dev), _ints([new] * 3, dev), table, kc, vc, max_new=new,
                        block_size=size, k_scale=ks, v_scale=vs, dev_status=st,
                        rope_table=_table(dev, R)[0] if R else None)
    assert int(st) == 0
    written = np.zeros((pool.pages, size), bool)
    grouped = np.zeros((pool.pages, size // kv.GROUP), bool)
    for b, n in enumerate(lens):
        for p in range(n, n + new):
            written[pool.table[b, p // size], p % size] = True
            grouped[pool.table[b, p // size], p % size // kv.GROUP] |= p // kv.GROUP > (n - 1) // kv.GROUP
    for got, was, scale, scale_was in zip((kc, vc), pool.codes, (ks, vs), pool.scale):
        same = torch.from_numpy(~written)[:, None, :, None].expand(was.shape)
        assert torch.equal(got.view(u8).cpu()[same], was[same])
        same = torch.from_numpy(~grouped)[:, None].expand(scale_was.shape)   # (groups begun anew get their own)
        assert torch.equal(scale.cpu()[same], scale_was[same])
