"""Drafted tokens through the whole loop, as they would be used: placed, run through the KDA
layer and the attention, accepted, given back, forked.

KDA: the tree's outputs and states against the same tokens one by one, both in fp32 arithmetic.
A value is a sum over 128 channels and, in the tree, over at most 24 updates of a path, each a
product off by 2^-24: by norm at most (128 + 24) 2^-24 = 9e-6 a token, and a state carries the
errors of the tokens before it, decayed; 24 of them at full weight give 2.2e-4.  Attention: the
outputs are bf16, off by at most 2^-8 of themselves; weights (16 bits) add 2^-16 of the values,
which the outputs, averages of them, fall below by less than the square root of 250 tokens."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("max_nodes,seed", [(24, 1), (7, 2), (1, 3)])
def test_drafted_tokens_serving_loop(lib, max_nodes, seed):
    spec = importlib.util.spec_from_file_location("draft_decode",
                                                  os.path.join(ROOT, "examples", "draft_decode.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    kda, attention = example.serve(steps=8, max_nodes=max_nodes, seed=seed)
    assert kda <= 2.2e-4
    assert attention <= 2.0 ** -8 + 16 * 2.0 ** -16
