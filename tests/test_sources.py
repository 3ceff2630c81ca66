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
