"""The serving example: KDA by state slot and attention over the paged cache in one loop.
bf16 outputs are rounded by at most 2^-8 of themselves; the rest is fp32 arithmetic."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("fp8", [False, True])
def test_hybrid_serving_loop(lib, fp8):
    spec = importlib.util.spec_from_file_location("hybrid_decode",
                                                  os.path.join(ROOT, "examples", "hybrid_decode.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    assert example.serve(steps=10, fp8=fp8, seed=3) <= 2.0 ** -8
