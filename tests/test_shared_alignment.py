"""Shared arrays of the paged kernels that are read or written as 16-byte vectors declare that
alignment (CPU: the sources are read; an array of a smaller type is only sure of its own)."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "gated_delta_rule_33_gb300", "csrc")
SOURCES = sorted(glob.glob(os.path.join(CSRC, "kda_page*.cu*")))
VECTOR = {"int2": 8, "uint2": 8, "float2": 8, "int4": 16, "uint4": 16, "float4": 16}


def declared_alignment(text, name):
    """Bytes that the shared declaration of `name` is sure of."""
    for m in re.finditer(r"__shared__([^;]*);", text):
        if not re.search(r"\b%s\s*\[" % name, m.group(1)):
            continue
        align = re.search(r"__align__\((\d+)\)", m.group(1))
        if align:
            return int(align.group(1))
        return VECTOR.get(m.group(1).split()[0], 4)
    raise AssertionError(f"no shared declaration of {name}")


@pytest.mark.parametrize("path", SOURCES, ids=os.path.basename)
def test_vector_access_to_shared_arrays(path):
    text = open(path).read()
    for m in re.finditer(r"reinterpret_cast<(?:const )?(\w+) \*>\(\s*&?(s_\w+)(?![\w]|\[\w+\]\.)", text):
        if m.group(1) in VECTOR:
            assert declared_alignment(text, m.group(2)) >= VECTOR[m.group(1)], m.group(0)


def test_the_sources_are_there():
    assert len(SOURCES) >= 6
