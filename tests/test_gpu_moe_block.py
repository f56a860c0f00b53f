"""The example block: one training step through the library against autograd in binary32.

What separates the two is the quantization: an FP8 cast to E4M3 is off by at most 2^-4 of a value,
in the root mean square 2^-4 / sqrt(3) = 3.6 % at worst (values at the low end of a binade) and
about 2.6 % on average.  Outputs pass through two casts (input, activations) and one bf16 rounding of
each product, gradients through the checkpoint on both factors as well: four casts, each with its own
independent rounding, 2 x 3.6 % in the root of the sum of squares.  The residual stream itself is not
quantized, so it is nearer.  Bound: 10 %."""
from __future__ import annotations

import os
import sys

import pytest

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.parametrize("tokens,channels,hidden,experts,k", [
    (512, 512, 256, 8, 2), (301, 640, 384, 12, 4), (1, 256, 128, 4, 2), (64, 256, 128, 40, 1)])
def test_training_step(cuda_device, tokens, channels, hidden, experts, k):
    import __graft_entry__
    __graft_entry__.build()
    import moe_block
    errors, saved = moe_block.step(tokens, channels, hidden, experts, k)
    assert sum(saved["sizes"]) == tokens * k
    # The router's gradient is made of differences of the experts' weight gradients, which may cancel
    # (with one expert they do exactly), so its error has no bound relative to itself; it is checked
    # against its formula in test_gpu_route.
    assert errors.pop("d router") >= 0
    for name, e in errors.items():
        assert e < 0.10, f"{name}: {e:.3f}"
