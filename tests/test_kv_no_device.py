"""Well-formed calls of the 8-bit cache's entry points where no device can be asked: an error status, in a process that lives.

The calls run in a process of their own that sees no GPU, on any machine: their pointers stand for nothing.
"""
import os
import subprocess
import sys

import pytest

from tests._util import ROOT, built_lib

ERR_CUDA = 5
PROGRAM = """
import ctypes
from eagle_tree_speculative_spec_gb300 import _lib as B
from tests import test_kv_abi as abi
L = B.lib()
print("status", {call})
"""


def _status(call):
    built_lib()
    env = dict(os.environ, CUDA_VISIBLE_DEVICES="-1", PYTHONPATH=ROOT)
    r = subprocess.run([sys.executable, "-c", PROGRAM.format(call=call)], env=env, cwd=ROOT, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0, (r.returncode, r.stderr[-500:])
    return int(r.stdout.split("status")[1])


@pytest.mark.parametrize("call", [
    "L.eagle3_rope_table(ctypes.byref(abi._table()), None)",
    "L.eagle3_rope(ctypes.byref(abi._rope()), None)",
    "L.eagle3_rope(ctypes.byref(abi._rope(rows=100000, elem_bytes=4, rotary_dim=20)), None)",
    "L.eagle3_append_kv(ctypes.byref(abi._append()), None)",
    "L.eagle3_append_kv(ctypes.byref(abi._append(max_new=100, n_rows=200)), None)",
    "L.eagle3_append_kv(ctypes.byref(abi._append(format=0)), None)",
    "L.eagle3_verify_attn_fp8(ctypes.byref(abi._attn(num_splits=1)), None, 0, None)"])
def test_no_device_is_an_error(call):
    assert _status(call) == ERR_CUDA


@pytest.mark.parametrize("kw", [
    "dict(n_rows=0, k_new=None, v_new=None)", "dict(n_rows=0, k_new=None, v_new=None, row_start=16)",
    "dict(n_rows=0, k_new=None, v_new=None, row_ids=16, rows_per_seq=5, n_new=None)", "dict(n_rows=0)"])
def test_an_append_of_no_rows_is_taken(kw):
    """An empty tensor has no address; whether a sequence has new tokens is known on the device only."""
    assert _status(f"L.eagle3_append_kv(ctypes.byref(abi._append(**{kw})), None)") == ERR_CUDA


@pytest.mark.parametrize("kw", ["dict(k_new=None)", "dict(n_rows=0, k_new=24)", "dict(n_rows=0, k_new=None, v_cache=None)"])
def test_an_append_without_its_tensors_is_refused(kw):
    assert _status(f"L.eagle3_append_kv(ctypes.byref(abi._append(**{kw})), None)") == 1
