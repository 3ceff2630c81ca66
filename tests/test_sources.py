"""Properties of the kernels' sources that no result shows: instructions that want a whole, converged warp stand behind a
__syncwarp() in their one helper, since a branch before them need not have come together again."""
import glob
import os
import re

import pytest

from tests._util import ROOT

CSRC = os.path.join(ROOT, "eagle_tree_speculative_spec_gb300", "csrc")


@pytest.mark.parametrize("instruction,uses", [("barrier.cluster", 1), ("setmaxnreg", 2)])
def test_aligned_instructions_are_converged(instruction, uses):
    found = 0
    for path in glob.glob(os.path.join(CSRC, "*.cu*")):
        text = open(path).read()
        for m in re.finditer(r'asm volatile\(\s*"[^;]*' + re.escape(instruction), text):
            found += 1
            body = text[text.rindex("E3_DEV void", 0, m.start()):m.start()]
            assert "}" not in body and "__syncwarp();" in body, (os.path.basename(path), body)
    assert found == uses


def test_other_ctas_are_told_at_cluster_scope():
    """What one CTA of a pair announces to the other about its shared memory is released and acquired at cluster scope;
    arrivals of the default scope announce TMEM reads only (tempty)."""
    tc = open(os.path.join(CSRC, "tc.cuh")).read()
    arrive = tc[tc.index("E3_DEV void mbar_arrive_cluster_smem"):tc.index("E3_DEV bool mbar_wait_cluster_smem")]
    wait = tc[tc.index("E3_DEV bool mbar_wait_cluster_smem"):]
    assert arrive.index("fence.release.sync_restrict::shared::cta.cluster") < arrive.index("mbarrier.arrive.relaxed.cluster")
    assert wait.index("try_wait.parity.relaxed.cluster") < wait.index("fence.acquire.sync_restrict::shared::cluster.cluster")
    for path in glob.glob(os.path.join(CSRC, "*.cu")):
        for line in open(path):
            if "mbar_arrive_cluster_if" in line:
                assert "tempty" in line, (os.path.basename(path), line)
