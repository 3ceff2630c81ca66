"""Host-side refusals of the 8-bit cache's entry points (no GPU needed)."""
import ctypes

import pytest
import torch

import eagle_tree_speculative_spec_gb300 as e3
from eagle_tree_speculative_spec_gb300 import _lib as B
from tests._util import built_lib

NAN, INF = float("nan"), float("inf")


def _table(**kw):
    base = dict(rotary_dim=128, scaling=0, original_positions=8192, theta=500000.0, factor=8.0, low_turns=1.0,
                high_turns=4.0, table=16)
    base.update(kw)
    return B.RopeTableArgs(**base)


@pytest.mark.parametrize("kw", [
    dict(rotary_dim=0), dict(rotary_dim=7), dict(rotary_dim=258), dict(scaling=-1), dict(scaling=5), dict(theta=1.0),
    dict(theta=NAN), dict(theta=INF), dict(scaling=1, factor=0.5), dict(scaling=1, factor=NAN),
    dict(scaling=1, factor=INF), dict(scaling=2, rotary_dim=2), dict(scaling=3, original_positions=0),
    dict(scaling=3, low_turns=0.0), dict(scaling=4, high_turns=1.0), dict(scaling=4, high_turns=INF), dict(table=None),
    dict(table=20)])
def test_table_refusals(kw):
    assert built_lib().eagle3_rope_table(ctypes.byref(_table(**kw)), None) == 1


def _rope(**kw):
    base = dict(rows=3, n_heads=2, head_dim=64, rotary_dim=64, elem_bytes=2, layout=0, inverse=0, amplitude=1.0,
                x_row_stride=0, out_row_stride=0, x=16, positions=16, table=16, out=32)
    base.update(kw)
    return B.RopeArgs(**base)


@pytest.mark.parametrize("kw,want", [
    (dict(rows=0), 0),
    (dict(rows=-1), 1),
    (dict(n_heads=0), 1),
    (dict(head_dim=60), 2),
    (dict(head_dim=264), 2),
    (dict(elem_bytes=1), 2),
    (dict(rotary_dim=66), 1),
    (dict(rotary_dim=3), 1),
    (dict(rotary_dim=0), 1),
    (dict(layout=2), 1),
    (dict(inverse=2), 1),
    (dict(amplitude=NAN), 1),
    (dict(x_row_stride=120), 1),             # rows overlap
    (dict(x_row_stride=132), 1),             # not 16 bytes
    (dict(out_row_stride=132), 1),
    (dict(elem_bytes=4, x_row_stride=130), 1),
    (dict(x=24), 1),
    (dict(out=None), 1),
    (dict(positions=18), 1),
    (dict(table=20), 1),
    (dict(out=16, out_row_stride=256), 1),   # in place at another pitch
    (dict(rows=2 ** 31 - 1), 2),
    (dict(n_heads=2 ** 30), 2),
])
def test_rope_refusals(kw, want):
    assert built_lib().eagle3_rope(ctypes.byref(_rope(**kw)), None) == want


def _append(**kw):
    base = dict(batch=2, n_kv_heads=2, head_dim=64, format=1, n_rows=10, max_new=5, rows_per_seq=0, max_blocks=3,
                block_size=64, n_pages=7, rotary_dim=64, rope_layout=0, rope_amplitude=1.0, row_stride=0, k_new=16,
                v_new=16, cache_len=16, n_new=16, row_start=None, row_ids=None, block_table=16, rope_table=16,
                k_cache=16, v_cache=16, k_scale=1, v_scale=1, dev_status=None)
    base.update(kw)
    return B.AppendKvArgs(**base)


@pytest.mark.parametrize("kw,want", [
    (dict(batch=0), 0),
    (dict(max_new=0), 0),
    (dict(batch=-1), 1),
    (dict(batch=65536), 2),
    (dict(n_kv_heads=0), 1),
    (dict(n_kv_heads=32768), 2),
    (dict(head_dim=60, rotary_dim=60), 2),
    (dict(head_dim=264, rotary_dim=64), 2),
    (dict(format=2), 1),
    (dict(n_rows=-1), 1),
    (dict(max_new=-1), 1),
    (dict(max_blocks=0), 1),
    (dict(block_size=0), 1),
    (dict(block_size=96), 1),                # not whole groups
    (dict(n_pages=0), 1),
    (dict(max_blocks=2 ** 25, block_size=128), 2),
    (dict(batch=65535, max_new=2 ** 20, max_blocks=2 ** 14), 2),   # more (group, head) jobs than 31 bits count
    (dict(rotary_dim=66), 1),
    (dict(rotary_dim=1), 1),
    (dict(rope_layout=-1), 1),
    (dict(rope_amplitude=INF), 1),
    (dict(row_stride=120), 1),
    (dict(row_stride=132), 1),
    (dict(n_new=None), 1),                   # without row ids
    (dict(row_ids=16), 1),                   # without rows_per_seq
    (dict(row_ids=16, rows_per_seq=5, row_start=16), 1),
    (dict(k_new=24), 1),
    (dict(v_cache=None), 1),
    (dict(k_scale=None), 1),
    (dict(cache_len=None), 1),
    (dict(block_table=18), 1),
    (dict(n_new=18), 1),
    (dict(rope_table=20), 1),
])
def test_append_refusals(kw, want):
    assert built_lib().eagle3_append_kv(ctypes.byref(_append(**kw)), None) == want


def _attn(**kw):
    base = dict(batch=2, n_nodes=3, n_heads=8, n_kv_heads=2, head_dim=128, max_prefix_len=100, num_splits=0, max_blocks=2,
                block_size=64, n_pages=9, sm_scale=0.0, q_node_stride=0, kv_node_stride=0, q=16, tree_k=None, tree_v=None,
                parents=None, k_cache=16, v_cache=16, k_scale=1, v_scale=1, block_table=16, prefix_len=16, out=16,
                lse=None, dev_status=None)
    base.update(kw)
    return B.VerifyAttnFp8Args(**base)


@pytest.mark.parametrize("kw,want", [
    (dict(batch=0), 0),
    (dict(batch=-1), 1),
    (dict(batch=65536), 2),
    (dict(n_nodes=0), 1),
    (dict(n_nodes=65), 2),
    (dict(n_heads=7), 1),
    (dict(n_heads=0), 1),
    (dict(n_heads=8192, n_kv_heads=2), 2),
    (dict(head_dim=64), 2),
    (dict(max_prefix_len=-1), 1),
    (dict(max_prefix_len=129), 3),
    (dict(num_splits=-1), 1),
    (dict(block_size=32), 1),
    (dict(max_blocks=0), 1),
    (dict(n_pages=0), 1),
    (dict(n_pages=2 ** 25, block_size=64), 2),
    (dict(sm_scale=-1.0), 1),
    (dict(sm_scale=NAN), 1),
    (dict(sm_scale=INF), 1),
    (dict(q_node_stride=1020), 1),
    (dict(q_node_stride=1028), 1),
    (dict(tree_k=16), 1),                    # a tree is three things
    (dict(tree_k=16, tree_v=16), 1),
    (dict(parents=16), 1),
    (dict(tree_k=24, tree_v=16, parents=16), 1),
    (dict(tree_k=16, tree_v=16, parents=16, kv_node_stride=130), 1),
    (dict(q=None), 1),
    (dict(k_cache=8), 1),
    (dict(v_scale=None), 1),
    (dict(prefix_len=None), 1),
    (dict(lse=18), 1),
    (dict(num_splits=2), 6),                 # without its workspace
])
def test_attn_refusals(kw, want):
    assert built_lib().eagle3_verify_attn_fp8(ctypes.byref(_attn(**kw)), None, 0, None) == want


def test_workspace_size():
    L = built_lib()
    size = lambda **kw: L.eagle3_verify_attn_fp8_workspace_size(ctypes.byref(_attn(**kw)))
    assert size(batch=0) == 0 and size(batch=-1) == 0 and size(num_splits=1) == 0
    assert size(num_splits=2) >= 2 * 2 * 3 * 8 * 130 * 4
    assert L.eagle3_verify_attn_fp8_workspace_size(None) == 0


def test_null_arguments():
    L = built_lib()
    assert L.eagle3_rope_table(None, None) == 1 and L.eagle3_rope(None, None) == 1
    assert L.eagle3_append_kv(None, None) == 1 and L.eagle3_verify_attn_fp8(None, None, 0, None) == 1


def test_binding_refuses_what_the_c_call_cannot_see():
    bf, f8, i32, i64, u8 = torch.bfloat16, torch.float8_e4m3fn, torch.int32, torch.int64, torch.uint8
    z = torch.zeros
    rope = lambda x=z(4, 2, 64), pos=z(4, dtype=i32), t=z(32, dtype=i64), out=z(4, 2, 64): e3.eagle3_rope(x, pos, t, out)
    with pytest.raises(ValueError, match="CUDA"):
        rope()
    for kw in (dict(pos=z(3, dtype=i32)), dict(out=z(4, 3, 64)), dict(x=z(4, 64, 2).transpose(1, 2)),
               dict(x=z(1, 2, 64).expand(4, 2, 64)), dict(t=z(8, 4, dtype=i64))):
        with pytest.raises(ValueError):
            rope(**kw)
    for kw in (dict(pos=z(4, dtype=i64)), dict(out=z(4, 2, 64, dtype=bf)), dict(x=z(4, 2, 64, dtype=torch.float16)),
               dict(t=z(32))):
        with pytest.raises(TypeError):
            rope(**kw)

    def append(k=z(6, 2, 64, dtype=bf), v=z(6, 2, 64, dtype=bf), n=z(2, dtype=i32), kc=z(3, 2, 64, 64, dtype=u8).view(f8),
               vc=z(3, 2, 64, 64, dtype=u8).view(f8), ks=z(3, 2, 1, dtype=u8), vs=z(3, 2, 1, dtype=u8), size=64, **kw):
        e3.eagle3_append_kv(k, v, z(2, dtype=i32), n, z(2, 4, dtype=i32), kc, vc, max_new=3, block_size=size, k_scale=ks,
                            v_scale=vs, **kw)
    with pytest.raises(ValueError, match="CUDA"):
        append()
    for kw in (dict(v=z(6, 3, 64, dtype=bf)), dict(v=z(6, 4, 64, dtype=bf)[:, :2]), dict(n=z(3, dtype=i32)),
               dict(ks=z(3, 2, 2, dtype=u8)), dict(vs=None), dict(size=128), dict(size=32), dict(size=0),
               dict(kc=z(192, 2, 64, dtype=bf), vc=z(192, 2, 64, dtype=bf)), dict(row_ids=z(2, 4, dtype=i32))):
        with pytest.raises(ValueError):
            append(**kw)
    for kw in (dict(k=z(6, 2, 64)), dict(ks=z(3, 2, 1)), dict(vc=z(3, 2, 64, 64, dtype=u8)), dict(rope_table=z(32))):
        with pytest.raises(TypeError):
            append(**kw)

    def attn(q=z(2, 3, 8, 128, dtype=bf), kc=z(5, 2, 64, 128, dtype=u8).view(f8), ks=z(5, 2, 1, dtype=u8),
             out=z(2, 3, 8, 128, dtype=bf), L=z(2, dtype=i32), **kw):
        e3.eagle3_verify_attn_fp8(q, kc, kc, ks, ks, z(2, 4, dtype=i32), L, out, max_prefix_len=100, **kw)
    with pytest.raises(ValueError, match="CUDA"):
        attn()
    tk, par = z(2, 3, 2, 128, dtype=bf), z(2, 3, dtype=i32)
    for kw in (dict(q=z(2, 8, 3, 128, dtype=bf).transpose(1, 2)), dict(ks=z(5, 2, 2, dtype=u8)), dict(L=z(3, dtype=i32)),
               dict(out=z(2, 3, 4, 128, dtype=bf)), dict(tree_k=tk), dict(tree_k=tk, tree_v=tk), dict(parents=par),
               dict(tree_k=tk, tree_v=z(2, 3, 4, 128, dtype=bf)[:, :, :2], parents=par), dict(lse=z(2, 3, 4))):
        with pytest.raises(ValueError):
            attn(**kw)
    for kw in (dict(q=z(2, 3, 8, 128)), dict(kc=z(5, 2, 64, 128, dtype=u8)), dict(L=z(2, dtype=i64)),
               dict(lse=z(2, 3, 8, dtype=bf))):
        with pytest.raises(TypeError):
            attn(**kw)
