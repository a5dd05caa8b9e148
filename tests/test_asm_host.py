"""What the compiler may not move is told to it: an instruction that the threads of a warp
carry out together is a volatile statement, so that none of them is left out of it.
And a kernel that starts while the preceding one runs does not read what that one may
write by the path for memory that stays as it is."""
import glob
import os
import re

import pytest

from split_kv_mla_gb300 import build as mla_build

SOURCES = sorted(glob.glob(os.path.join(mla_build.CSRC, "*.cu*")) +
                 glob.glob(os.path.join(mla_build.CSRC, "*.h")) +
                 glob.glob(os.path.join(mla_build.HERE, "probes", "*.cu")))


@pytest.mark.parametrize("path", SOURCES, ids=os.path.basename)
def test_collective_instructions_are_volatile(path):
    with open(path) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    for m in re.finditer(r"\basm\s*(volatile)?\s*\(\s*((?:\"[^\"]*\"\s*)+)", text):
        if re.search(r"\.sync\b|griddepcontrol|mbarrier", m.group(2)):
            assert m.group(1), m.group(2)


def test_step_kernels_read_coherently():
    with open(os.path.join(mla_build.CSRC, "mla_step.cu")) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    assert "wait_for_predecessor()" in text
    assert "__ldg" not in text and "global.nc" not in text and "__restrict__" not in text
