"""examples/decoder_block.py: the operators together against the block in 64
bits.  fp16 storage between the operators costs half a unit (2^-11) in each of
a handful of tensors, and fake-quantized weights (fp16) another in the expert
products: 2e-3 of the outputs' norm covers them, with 8-bit codes that sit on
the other side of a rounding boundary in rare elements."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "decoder_block.py")


@pytest.mark.parametrize("tokens", [1, 7, 64])
def test_decoder_block(gpu, tokens):
    spec = importlib.util.spec_from_file_location("decoder_block", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    assert m.main(["--tokens", str(tokens), "--check"]) <= 2e-3
