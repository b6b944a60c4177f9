"""examples/cached_attention.py: prompts, beams, reordering and compaction against attention in 64 bits on
unquantized keys and values.

What 8 bits cost is the whole difference, relative to the output's norm.  A code is off by up to half a step of
the block's largest value / 127; these blocks (16 tokens of 64 channels) have largest values of some 3.5 times their
spread, so an error of 3.5 / 127 / sqrt(12) = 0.8 % of the spread in v, as much in k (times the scores' spread,
which is about 1), and both once more for every time a block's scale grows and its codes are rounded again (a
handful, each smaller).  The codes of the activations in front of the two projections add 1 / 127 of their own
largest values, 0.8 % each.  Five such parts in quadrature are 1.8 %; 5e-2 leaves room for their ends.
"""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "cached_attention.py")


@pytest.mark.parametrize("steps", [0, 1, 12])
def test_cached_attention(gpu, steps):
    spec = importlib.util.spec_from_file_location("cached_attention", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    assert m.main(["--steps", str(steps), "--check"]) <= 5e-2
