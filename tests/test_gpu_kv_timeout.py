"""The timeout path of the 8-bit cache's attention, on the GPU, without a fault or a hang.

The test hook (include/eagle3_testing.h) lets the barrier of one load stage expect an arrival that never comes and
limits every wait to about a millisecond.  Checked: the call returns within its limits, the status word carries
EAGLE3_DEV_TIMEOUT, and the same context then gives the bits that it gave before.  The kernel of 16 rows has no waits.
"""
import ctypes
import time

import numpy as np
import pytest
import torch

from eagle_tree_speculative_spec_gb300 import _lib
from tests._util import built_lib, require_gpu

LIMIT = 2_000_000   # clocks, about 1 ms
bf, i32, u8, f8 = torch.bfloat16, torch.int32, torch.uint8, torch.float8_e4m3fn


def _inputs(dev, lens, N, Hq, Hkv, size, tree):
    g = torch.Generator().manual_seed(N + sum(lens))
    need = [-(-n // size) for n in lens]
    table = torch.full((len(lens), max(need)), -1, dtype=i32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = torch.arange(at, at + n, dtype=i32)
        at += n
    caches = [torch.randn(at, Hkv, size, 128, generator=g).mul_(60).to(f8).to(dev) for _ in range(2)]
    scales = [torch.full((at, Hkv, size // 64), 120, dtype=u8, device=dev) for _ in range(2)]
    q, tk, tv = (torch.randn(len(lens), N, h, 128, generator=g).to(bf).to(dev) for h in (Hq, Hkv, Hkv))
    par = torch.from_numpy(np.maximum(np.arange(N) - 2, np.minimum(np.arange(N) - 1, 0)).astype(np.int32))
    out, st = torch.empty_like(q), torch.zeros(1, dtype=i32, device=dev)
    kw = dict(max_prefix_len=max(lens), dev_status=st)
    if tree:
        kw.update(tree_k=tk, tree_v=tv, parents=par.repeat(len(lens), 1).to(dev))
    return (q, *caches, *scales, table.to(dev), torch.tensor(lens, dtype=i32, device=dev), out), kw


@pytest.mark.gpu
@pytest.mark.parametrize("lens,N,Hq,tree,splits,stall", [
    (*c, stall) for c in (([900], 20, 2, False, 1), ([900], 20, 2, True, 1), ([2000, 0, 700], 60, 8, True, 1),
                          ([4000] * 40, 60, 8, True, 0)) for stall in (0, 1, 3)] +
    [([2000, 0, 700], 60, 8, True, 0, 0)])   # (CTAs of two tiles)
def test_waits_run_out(lens, N, Hq, tree, splits, stall):
    dev = require_gpu()
    args, kw = _inputs(dev, lens, N, Hq, 1, 64, tree)
    out, st = args[-1], kw["dev_status"]
    kw["num_splits"] = splits
    hook = _lib.eagle3_test_verify_attn_fp8
    hook(*args, kernel=2, **kw)
    torch.cuda.synchronize()
    assert int(st) == 0
    want = out.clone()
    t0 = time.monotonic()
    hook(*args, kernel=2, stall_block=stall, wait_limit_cycles=LIMIT, **kw)
    torch.cuda.synchronize()
    took = time.monotonic() - t0
    assert int(st) == _lib.DEV_TIMEOUT and took < 1.0, (int(st), took)
    st.zero_()
    for _ in range(2):
        out.zero_()
        hook(*args, kernel=2, **kw)
        torch.cuda.synchronize()
        assert int(st) == 0 and torch.equal(out, want)


@pytest.mark.parametrize("kernel,stall,limit", [(0, -1, 0), (3, -1, 0), (1, 0, 10_000), (2, -2, 10_000), (2, 4, 10_000),
                                                (2, 0, 10), (2, 0, 10**10)])
def test_hook_refuses(kernel, stall, limit):
    L, a = built_lib(), _lib.VerifyAttnFp8Args()
    assert L.eagle3_test_verify_attn_fp8(ctypes.byref(a), None, 0, kernel, stall, limit, None) == 1
    assert kernel in (1, 2) or L.eagle3_test_verify_attn_fp8_workspace_size(ctypes.byref(a), kernel) == 0
