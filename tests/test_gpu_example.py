"""The example layer runs and stays near plain PyTorch on the same weights.

What differs from plain there is the rounding of activations to e4m3 (3
mantissa bits: relative error at most 2^-4 a value, below 2^-5 in the 2-norm),
before each of the two products of the shared expert, and before the head: at
most 3 * 2^-5 in all, with what 16-bit results add (2^-8)."""
import os
import sys

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def test_moe_layer():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import moe_layer
    for n, out, logits, us in moe_layer.run([1, 5, 40], hidden=512, inter=256, shared=384, experts=8, top_k=2, vocab=1000,
                                            replays=4):
        assert out < 3 * 2.0 ** -5 + 2.0 ** -8 and logits < 3 * 2.0 ** -5 + 2.0 ** -8, (n, out, logits)
