"""Host-side refusals of the mixture-of-experts and 8-bit entry points (no GPU needed)."""
import ctypes
import os
import shutil
import subprocess

import pytest
import torch

import eagle_tree_speculative_spec_gb300 as e3
from eagle_tree_speculative_spec_gb300 import _lib as B
from tests._util import ROOT, built_lib


def _route(**kw):
    base = dict(rows=40, n_experts=16, top_k=4, scoring=0, renormalize=1, scale=1.0, ld_logits=0, logits=16,
                num_rows=None, topk_ids=16, topk_weights=16, expert_offsets=16, sorted_rows=16, slots=16,
                dev_status=None)
    base.update(kw)
    return B.MoeRouteArgs(**base)


@pytest.mark.parametrize("kw,want", [
    (dict(rows=-1), 1),
    (dict(n_experts=0), 1),
    (dict(n_experts=513), 2),
    (dict(top_k=0), 1),
    (dict(top_k=17, n_experts=32), 2),
    (dict(top_k=5, n_experts=4), 1),
    (dict(scoring=2), 1),
    (dict(renormalize=2), 1),
    (dict(scale=float("nan")), 1),
    (dict(scale=float("inf")), 1),
    (dict(ld_logits=15), 1),
    (dict(rows=2 ** 30), 2),                 # more slots than 32 bits count
    (dict(rows=2 ** 31 - 70000, top_k=1), 2),   # rows of whole blocks pass 32 bits
    (dict(logits=None), 1),
    (dict(slots=None), 1),
    (dict(rows=0, expert_offsets=None), 1),  # the offsets are written for no rows too
    (dict(topk_ids=18), 1),
    (dict(rows=257), 6),                     # from 257 rows on with a workspace
])
def test_route_refusals(kw, want):
    a = _route(**kw)
    assert built_lib().eagle3_moe_route(ctypes.byref(a), None, 0, None) == want


def test_route_workspace_size():
    L = built_lib()
    size = lambda **kw: L.eagle3_moe_route_workspace_size(ctypes.byref(_route(**kw)))
    assert size(rows=0) == 0 and size(rows=32) == 0 and size(rows=256) == 0
    assert size(rows=257) == 9 * 16 * 4
    assert size(rows=200000) <= 152 * 16 * 4
    assert size(rows=-1) == 0
    assert L.eagle3_moe_route_workspace_size(None) == 0


def _grouped(**kw):
    base = dict(n_groups=4, m=10, n=64, k=128, n_src=5, epilogue=0, ld_x=0, ld_w=0, ld_out=0, x=16, w=16, w2=None,
                out=16, offsets=16, row_ids=None, dev_status=None)
    base.update(kw)
    return B.GroupedLinearArgs(**base)


@pytest.mark.parametrize("kw,want", [
    (dict(m=0), 0),
    (dict(m=-1), 1),
    (dict(n_groups=0), 1),
    (dict(n_groups=513), 2),
    (dict(n=0), 1),
    (dict(k=0), 1),
    (dict(k=12), 2),
    (dict(epilogue=-1), 1),
    (dict(epilogue=5), 1),
    (dict(epilogue=1), 2),                   # fp32, residual and RoPE outputs are not offered
    (dict(epilogue=2), 2),
    (dict(epilogue=4), 2),
    (dict(epilogue=3), 1),                   # SwiGLU without w2
    (dict(row_ids=16, n_src=0), 1),
    (dict(ld_x=120), 1),
    (dict(ld_x=132), 1),
    (dict(ld_out=63), 1),
    (dict(x=None), 1),
    (dict(w=24), 1),
    (dict(out=17), 1),
    (dict(offsets=None), 1),
    (dict(offsets=18), 1),
    (dict(m=2 ** 31 - 1, n=2 ** 31 - 1), 2),
])
def test_grouped_refusals(kw, want):
    a = _grouped(**kw)
    assert built_lib().eagle3_grouped_linear(ctypes.byref(a), None) == want


def _combine(**kw):
    base = dict(rows=4, n_slots=8, top_k=2, dim=64, ld_y=0, ld_res=0, ld_out=0, y=16, slots=16, weights=16,
                residual=None, out=16, dev_status=None)
    base.update(kw)
    return B.MoeCombineArgs(**base)


@pytest.mark.parametrize("kw,want", [
    (dict(rows=0), 0),
    (dict(rows=-1), 1),
    (dict(n_slots=-1), 1),
    (dict(top_k=0), 1),
    (dict(top_k=17), 2),
    (dict(dim=0), 1),
    (dict(ld_y=63), 1),
    (dict(y=None), 1),
    (dict(out=None), 1),
    (dict(out=17), 1),
    (dict(slots=18), 1),
])
def test_combine_refusals(kw, want):
    a = _combine(**kw)
    assert built_lib().eagle3_moe_combine(ctypes.byref(a), None) == want


def _quantize(**kw):
    base = dict(rows=4, k=64, ld_x=0, ld_q=0, x=16, q=16, scale=16)
    base.update(kw)
    return B.QuantizeFp8Args(**base)


@pytest.mark.parametrize("kw,want", [
    (dict(rows=0), 0),
    (dict(rows=-1), 1),
    (dict(k=0), 1),
    (dict(k=24), 2),
    (dict(ld_x=56), 1),
    (dict(ld_x=68), 1),
    (dict(ld_q=72), 1),
    (dict(x=24), 1),
    (dict(q=8), 1),
    (dict(scale=18), 1),
    (dict(scale=None), 1),
])
def test_quantize_refusals(kw, want):
    a = _quantize(**kw)
    assert built_lib().eagle3_quantize_fp8(ctypes.byref(a), None) == want


def _fp8(**kw):
    base = dict(m=4, n=64, k=128, epilogue=0, ld_x=0, ld_w=0, ld_out=0, ld_res=0, x=16, x_scale=16, w=16, w_scale=16,
                w2=None, w2_scale=None, out=16, residual=None, dev_status=None)
    base.update(kw)
    return B.LinearFp8Args(**base)


@pytest.mark.parametrize("kw,want", [
    (dict(m=0), 0),
    (dict(m=-1), 1),
    (dict(n=0), 1),
    (dict(k=0), 1),
    (dict(k=120), 2),
    (dict(epilogue=-1), 1),
    (dict(epilogue=4), 2),
    (dict(epilogue=5), 1),
    (dict(epilogue=2), 1),                   # residual missing
    (dict(epilogue=3, w2=16), 1),            # w2_scale missing
    (dict(ld_x=112), 1),
    (dict(ld_w=136), 1),
    (dict(ld_out=60), 1),
    (dict(x=24), 1),
    (dict(w=None), 1),
    (dict(x_scale=18), 1),
    (dict(epilogue=1, out=18), 1),
])
def test_fp8_refusals(kw, want):
    a = _fp8(**kw)
    assert built_lib().eagle3_linear_fp8(ctypes.byref(a), None) == want


def test_null_arguments():
    L = built_lib()
    assert L.eagle3_moe_route(None, None, 0, None) == 1
    assert L.eagle3_grouped_linear(None, None) == 1
    assert L.eagle3_moe_combine(None, None) == 1
    assert L.eagle3_quantize_fp8(None, None) == 1
    assert L.eagle3_linear_fp8(None, None) == 1


def test_binding_refuses_what_the_c_call_cannot_see():
    """Types, shapes, strides and devices are checked before any pointer is taken."""
    bf, f8, i32 = torch.bfloat16, torch.float8_e4m3fn, torch.int32
    z = torch.zeros
    route = lambda logits=z(4, 8), ids=z(4, 2, dtype=i32), off=z(9, dtype=i32), srt=z(8, dtype=i32): \
        e3.eagle3_moe_route(logits, ids, z(4, 2), off, srt, z(4, 2, dtype=i32))
    for kw in (dict(off=z(8, dtype=i32)), dict(srt=z(7, dtype=i32)), dict(ids=z(3, 2, dtype=i32))):
        with pytest.raises(ValueError):
            route(**kw)
    with pytest.raises(TypeError):
        route(logits=z(4, 8, dtype=bf))
    with pytest.raises(ValueError, match="CUDA"):
        route()
    w, off = z(3, 16, 8, dtype=bf), z(4, dtype=i32)
    with pytest.raises(ValueError):
        e3.eagle3_grouped_linear(z(5, 8, dtype=bf), w, off, z(6, 16, dtype=bf))      # x rows without row_ids
    with pytest.raises(ValueError):
        e3.eagle3_grouped_linear(z(6, 8, dtype=bf).t().contiguous().t(), w, off, z(6, 16, dtype=bf))
    with pytest.raises(ValueError, match="overlap"):
        e3.eagle3_grouped_linear(z(8, dtype=bf).expand(6, 8), w, off, z(6, 16, dtype=bf))
    with pytest.raises(TypeError):
        e3.eagle3_grouped_linear(z(6, 8, dtype=bf), w, z(4, dtype=torch.int64), z(6, 16, dtype=bf))
    with pytest.raises(ValueError):
        e3.eagle3_moe_combine(z(4, 8, dtype=bf), z(3, 2, dtype=i32), z(3, 2), z(3, 9, dtype=bf))
    with pytest.raises(ValueError):
        e3.eagle3_quantize_fp8(z(3, 144, dtype=bf), z(3, 144, dtype=f8), z(3, 2))     # scale is [k blocks, m]
    with pytest.raises(TypeError):
        e3.eagle3_quantize_fp8(z(3, 144, dtype=bf), z(3, 144, dtype=torch.uint8), z(2, 3))
    with pytest.raises(TypeError):
        e3.eagle3_linear_fp8(z(3, 144, dtype=f8), z(2, 3), z(5, 144, dtype=f8), z(1, 2), z(3, 5, dtype=bf),
                             epilogue=e3.EPI_F32)
    with pytest.raises(ValueError):
        e3.eagle3_linear_fp8(z(3, 144, dtype=f8), z(2, 3), z(5, 144, dtype=f8), z(2, 1), z(3, 5, dtype=bf))


C_SOURCE = r"""
#include "eagle3_moe.h"
#include "eagle3_fp8.h"

#include <string.h>

int main(void) {
    eagle3_moe_route_args_t r;
    eagle3_grouped_linear_args_t g;
    eagle3_moe_combine_args_t c;
    eagle3_quantize_fp8_args_t q;
    eagle3_linear_fp8_args_t f;
    memset(&r, 0, sizeof r);
    memset(&g, 0, sizeof g);
    memset(&c, 0, sizeof c);
    memset(&q, 0, sizeof q);
    memset(&f, 0, sizeof f);
    r.n_experts = EAGLE3_MOE_MAX_EXPERTS + 1;
    r.top_k = 1;
    r.scoring = EAGLE3_MOE_SIGMOID;
    if (eagle3_moe_route(&r, NULL, 0, NULL) != EAGLE3_ERR_UNSUPPORTED) return 1;
    if (eagle3_moe_route_workspace_size(&r) != 0) return 2;
    g.n_groups = g.n = 1;
    g.k = 8;
    if (eagle3_grouped_linear(&g, NULL) != EAGLE3_OK) return 3;
    c.top_k = c.dim = 1;
    if (eagle3_moe_combine(&c, NULL) != EAGLE3_OK) return 4;
    q.k = 16;
    if (eagle3_quantize_fp8(&q, NULL) != EAGLE3_OK) return 5;
    f.n = 1;
    f.k = 16;
    f.epilogue = EAGLE3_EPI_BF16_ROPE;
    if (eagle3_linear_fp8(&f, NULL) != EAGLE3_ERR_UNSUPPORTED) return 6;
    return 0;
}
"""


def test_headers_compile_as_c99_and_link(tmp_path):
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("no C compiler")
    libdir = os.path.dirname(built_lib()._name)
    src, exe = tmp_path / "abi.c", tmp_path / "abi"
    src.write_text(C_SOURCE)
    cmd = [gcc, "-std=c99", "-Wall", "-Wextra", "-Werror", "-pedantic", "-I", os.path.join(ROOT, "include"),
           str(src), "-o", str(exe), "-L", libdir, "-leagle3", "-Wl,-rpath," + libdir]
    res = subprocess.run(cmd, capture_output=True, text=True)
    assert res.returncode == 0, res.stderr
    assert subprocess.run([str(exe)], timeout=120).returncode == 0
