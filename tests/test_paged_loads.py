"""The paged kernels are set up while the kernel before them still writes what they read, so
they read by ordinary loads (CPU: the sources are read)."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "gated_delta_rule_33_gb300", "csrc")
SOURCES = sorted(glob.glob(os.path.join(CSRC, "kda_page*.cu*")))


@pytest.mark.parametrize("path", SOURCES, ids=os.path.basename)
def test_no_load_that_need_not_stay_behind_the_wait(path):
    code = re.sub(r"//[^\n]*", "", open(path).read())
    for unsafe in ("__ldg", "__ldcs", "__restrict__", "ld.global.nc"):
        assert unsafe not in code, unsafe
    # every kernel that is launched early waits
    kernels = re.findall(r"__global__ void.*?\n}\n", code, flags=re.S)
    for body in kernels:
        assert "wait_for_kernel_before();" in body


def test_the_sources_are_there():
    assert len(SOURCES) >= 6
