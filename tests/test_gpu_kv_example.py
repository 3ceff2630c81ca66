"""The 8-bit cache's usage example of the package's documentation, run as written: every output is finite and no device
error is reported."""
import pytest
import torch

import eagle_tree_speculative_spec_gb300 as e3
from tests._util import require_gpu

pytestmark = pytest.mark.gpu


def test_kv_usage_example():
    require_gpu()
    dev, bf, i32, u8, f8 = "cuda", torch.bfloat16, torch.int32, torch.uint8, torch.float8_e4m3fn
    B, Hq, Hkv, D, N, page, pages = 2, 32, 8, 128, 12, 64, 16      # 16 pages of 64 places
    ints = lambda *v: torch.tensor(v, dtype=i32, device=dev)
    k_cache, v_cache = torch.zeros(2, pages, Hkv, page, D, device=dev).to(f8)
    k_scale, v_scale = torch.ones(2, pages, Hkv, page // 64, dtype=u8, device=dev)
    blocks = torch.randperm(pages, device=dev).to(i32).view(B, -1)
    status = torch.zeros(1, dtype=i32, device=dev)
    turns = torch.empty(D // 2, dtype=torch.int64, device=dev)     # made once
    e3.eagle3_rope_table(turns, theta=500000.0, scaling=e3.ROPE_BANDS, factor=8.0)
    cache = dict(block_size=page, k_scale=k_scale, v_scale=v_scale, rope_table=turns, dev_status=status)

    prompt, length = ints(70, 129), ints(0, 0)
    k, v = torch.randn(2, 199, Hkv, D, device=dev).to(bf)          # the rows of both, one after the other
    e3.eagle3_append_kv(k, v, length, prompt, blocks, k_cache, v_cache, max_new=129, row_start=ints(0, 70), **cache)
    length += prompt
    k, v = torch.randn(2, B, Hkv, D, device=dev).to(bf)            # a token each
    e3.eagle3_append_kv(k, v, length, ints(1, 1), blocks, k_cache, v_cache, max_new=1, **cache)
    q = torch.randn(B, Hq, D, device=dev).to(bf)
    e3.eagle3_rope(q, length, turns, q)                            # in place, at the token's position
    length += 1
    out = torch.empty(B, 1, Hq, D, dtype=bf, device=dev)
    e3.eagle3_verify_attn_fp8(q[:, None], k_cache, v_cache, k_scale, v_scale, blocks, length, out, max_prefix_len=512)

    parents = torch.arange(-1, N - 1, dtype=i32, device=dev).repeat(B, 1)   # a chain; any tree with parents before children
    tq = torch.randn(B, N, Hq, D, device=dev).to(bf)               # tree queries and keys come rotated (or by eagle3_rope)
    tk, tv = torch.randn(2, B, N, Hkv, D, device=dev).to(bf)
    out = torch.empty_like(tq)
    e3.eagle3_verify_attn_fp8(tq, k_cache, v_cache, k_scale, v_scale, blocks, length, out, max_prefix_len=512,
                              tree_k=tk, tree_v=tv, parents=parents, dev_status=status)
    torch.cuda.synchronize()
    assert int(status) == 0
    assert torch.isfinite(out).all() and torch.isfinite(q).all()
    assert int(length[0]) == 71 and int(length[1]) == 130
