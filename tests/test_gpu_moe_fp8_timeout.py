"""The timeout paths of the grouped and the 8-bit products, on the GPU, without a fault or a hang.

The test hooks (include/eagle3_testing.h) let the barrier of one k-block expect an arrival that never comes, in every
CTA or in those of one rank of a cluster, and limit every wait to about a millisecond.  Checked, in every kernel variant: the call returns within its
limits, the status word carries EAGLE3_DEV_TIMEOUT, and the same context then gives the bits that it gave before.
"""
import time

import pytest
import torch

import eagle_tree_speculative_spec_gb300 as e3
from eagle_tree_speculative_spec_gb300 import _lib
from tests._util import built_lib, require_gpu

LIMIT = 2_000_000   # clocks, about 1 ms
bf, f32, i32, f8 = torch.bfloat16, torch.float32, torch.int32, torch.float8_e4m3fn


def _grouped_call(dev, counts, n, k, swiglu, gather):
    g = torch.Generator().manual_seed(n + k)
    m, E = sum(counts), len(counts)
    x, w, w2 = (torch.randn(*s, generator=g).to(bf).to(dev) for s in ((m, k), (E, n, k), (E, n, k)))
    off = torch.tensor([0] + list(torch.tensor(counts).cumsum(0)), dtype=i32, device=dev)
    ids = torch.arange(m, dtype=i32, device=dev) if gather else None
    out, st = torch.empty(m, n, dtype=bf, device=dev), torch.zeros(1, dtype=i32, device=dev)
    kw = dict(epilogue=e3.EPI_SWIGLU if swiglu else e3.EPI_BF16, w2=w2 if swiglu else None, row_ids=ids, dev_status=st)
    return (x, w, off, out), kw


def _fp8_call(dev, m, n, k, epi, out_pitch=0):
    g = torch.Generator().manual_seed(m + n + k)
    kb, nb = -(-k // 128), -(-n // 128)
    x, w, w2 = (torch.randn(*s, generator=g).to(f8).to(dev) for s in ((m, k), (n, k), (n, k)))
    xs, ws = torch.rand(kb, m, generator=g).to(dev), torch.rand(nb, kb, generator=g).to(dev)
    out = torch.zeros(m, n + out_pitch, dtype=f32 if epi == e3.EPI_F32 else bf, device=dev)[:, :n]
    swiglu, st = epi == e3.EPI_SWIGLU, torch.zeros(1, dtype=i32, device=dev)
    kw = dict(epilogue=epi, w2=w2 if swiglu else None, w2_scale=ws if swiglu else None, dev_status=st,
              residual=torch.randn(m, n, generator=g).to(bf).to(dev) if epi == e3.EPI_BF16_RESIDUAL else None)
    return (x, xs, w, ws, out), kw


def _gives_up(call, hook, args, kw, stall_block, stall_rank, limit=LIMIT, least=0.0, most=1.0):
    """hook(...) ends in time with the flag set; call(...) gives the same bits before and after."""
    out, st = args[-1], kw["dev_status"]
    call(*args, **kw)
    torch.cuda.synchronize()
    assert int(st) == 0
    want = out.clone()
    t0 = time.monotonic()
    hook(*args, stall_block=stall_block, stall_rank=stall_rank, wait_limit_cycles=limit, **kw)
    torch.cuda.synchronize()
    took = time.monotonic() - t0
    assert int(st) == _lib.DEV_TIMEOUT and least <= took < most, (int(st), took)
    st.zero_()
    for _ in range(2):
        out.zero_()
        call(*args, **kw)
        torch.cuda.synchronize()
        assert int(st) == 0 and torch.equal(out, want)


STALLS = [(0, -1), (2, -1), (1, 0), (1, 1)]   # (block, rank); rank 1 only where there are clusters
SINGLE = [([1], 128, 256, False), ([300, 7], 128, 640, False)]   # one weight tile: single CTAs
PAIRS = [([1], 128, 256, True), ([300, 7], 128, 640, True), ([300, 0, 90], 512, 640, False), ([300, 0, 90], 512, 640, True)]
SPLIT = [([2, 3], 128, 4096, False), ([2, 3], 128, 4096, True)]   # k over a cluster


@pytest.mark.gpu
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("counts,n,k,swiglu,stall_block,stall_rank",
                         [(*c, *s) for c in SINGLE for s in STALLS[:3]] + [(*c, *s) for c in PAIRS + SPLIT for s in STALLS])
def test_grouped_waits_run_out(counts, n, k, swiglu, gather, stall_block, stall_rank):
    args, kw = _grouped_call(require_gpu(), counts, n, k, swiglu, gather)
    _gives_up(e3.eagle3_grouped_linear, _lib.eagle3_test_grouped_linear_timeout, args, kw, stall_block, stall_rank)


ALONE = [(8, 128, 256, 0), (300, 512, 640, 0), (300, 512, 640, 1)]            # narrow; wide, outputs by TMA and by the warps
CLUSTERS = [(60, 200, 4096, 0), (200, 512, 8192, 0), (1100, 1001, 6160, 0)]   # narrow; wide, tiles of 128 and 256 columns


@pytest.mark.gpu
@pytest.mark.parametrize("epi", [e3.EPI_BF16, e3.EPI_F32, e3.EPI_BF16_RESIDUAL, e3.EPI_SWIGLU])
@pytest.mark.parametrize("m,n,k,out_pitch,stall_block,stall_rank",
                         [(*c, *s) for c in ALONE for s in ((0, -1), (1, -1), (1, 0))] +
                         [(*c, *s) for c in CLUSTERS for s in STALLS])
def test_fp8_waits_run_out(m, n, k, out_pitch, epi, stall_block, stall_rank):
    args, kw = _fp8_call(require_gpu(), m, n, k, epi, out_pitch)
    _gives_up(e3.eagle3_linear_fp8, _lib.eagle3_test_linear_fp8_timeout, args, kw, stall_block, stall_rank)


@pytest.mark.gpu
def test_longest_wait():
    """The library's own limit, 4e9 clocks: two seconds at 2 GHz, and as much again for the copies of a CTA whose
    barrier misses an arrival."""
    dev = require_gpu()
    args, kw = _grouped_call(dev, [300], 256, 1024, True, True)
    _gives_up(e3.eagle3_grouped_linear, _lib.eagle3_test_grouped_linear_timeout, args, kw, 1, -1, limit=4_000_000_000,
              least=1.5, most=12.0)
    args, kw = _fp8_call(dev, 300, 512, 1024, e3.EPI_BF16)
    _gives_up(e3.eagle3_linear_fp8, _lib.eagle3_test_linear_fp8_timeout, args, kw, 1, -1, limit=4_000_000_000,
              least=1.5, most=12.0)


@pytest.mark.parametrize("stall_block,stall_rank,limit", [(-1, -1, 10_000), (4, -1, 10_000), (0, -2, 10_000), (0, -1, 10), (0, -1, 10**10)])
def test_hooks_refuse_bad_limits(stall_block, stall_rank, limit):
    import ctypes
    L = built_lib()
    g, f = _lib.GroupedLinearArgs(), _lib.LinearFp8Args()
    g.n_groups, g.n, g.k, f.n, f.k = 1, 1, 8, 1, 16   # no rows
    assert L.eagle3_test_grouped_linear_timeout(ctypes.byref(g), stall_block, stall_rank, limit, None) == 1
    assert L.eagle3_test_linear_fp8_timeout(ctypes.byref(f), stall_block, stall_rank, limit, None) == 1
    assert L.eagle3_test_grouped_linear_timeout(ctypes.byref(g), 0, -1, 10_000, None) == 0
    assert L.eagle3_test_linear_fp8_timeout(ctypes.byref(f), 0, -1, 10_000, None) == 0
