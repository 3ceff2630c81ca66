"""Host-side values kept per device: a query that failed is asked again, one that succeeded is not (no GPU needed)."""
import os
import shutil
import subprocess

import pytest

from tests._util import ROOT

SOURCE = r"""
#include "common.cuh"

int main() {
    int asked = 0;
    e3::PerDevice<int> sms;
    auto count = [&] { return ++asked < 3 ? 0 : 152; };
    if (sms.get(count) != 0 || sms.get(count) != 0) return 1;
    if (sms.get(count) != 152 || sms.get(count) != 152 || asked != 3) return 2;
    asked = 0;
    e3::PerDevice<cudaError_t> attr;
    auto set = [&] { return ++asked < 2 ? cudaErrorMemoryAllocation : cudaSuccess; };
    if (attr.get(set) != cudaErrorMemoryAllocation || attr.get(set) != cudaSuccess) return 3;
    if (attr.get(set) != cudaSuccess || asked != 2) return 4;
    asked = 0;
    e3::PerDevice<e3::ClusterCounts> clusters;
    auto ask = [&] {
        e3::ClusterCounts c = {};
        c.n[2] = 76, c.n[7] = ++asked < 2 ? -1 : 0;   // a size that failed; none of that size fit
        return c;
    };
    if (e3::succeeded(clusters.get(ask)) || clusters.get(ask).n[7] != 0 || clusters.get(ask).n[2] != 76) return 5;
    return asked == 2 ? 0 : 6;
}
"""

# in place of the runtime's function: no GPU is needed
DEVICE = "int cudaGetDevice(int *device) { *device = 3; return 0; }\n"


def test_failed_queries_are_asked_again(tmp_path):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("no CUDA compiler")
    src, dev, exe = tmp_path / "per_device.cu", tmp_path / "device.c", tmp_path / "per_device"
    src.write_text(SOURCE)
    dev.write_text(DEVICE)
    csrc = os.path.join(ROOT, "eagle_tree_speculative_spec_gb300", "csrc")
    cmd = [nvcc, "-std=c++17", "-cudart", "shared", "--expt-relaxed-constexpr", "-gencode", "arch=compute_103a,code=sm_103a",
           "-I", csrc, "-I", os.path.join(ROOT, "include"), str(src), str(dev), "-o", str(exe), "-Xlinker", "-rpath", "-Xlinker",
           "/usr/local/cuda/lib64"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    assert res.returncode == 0, res.stderr
    assert subprocess.run([str(exe)], timeout=120).returncode == 0
