"""examples/experts.py: codes of weights, on the host."""
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def test_a_block_of_zeros_has_codes_and_scale_zero():
    import experts
    g = torch.Generator().manual_seed(1)
    w = torch.randn(2, 200, 300, generator=g)
    w[0, :128, 128:256] = 0
    w[1] = 0
    codes, scale = experts.codes_of(w)
    assert codes.shape == w.shape and scale.shape == (2, 2, 3)
    assert not codes[0, :128, 128:256].float().any() and scale[0, 0, 1] == 0
    assert not codes[1].float().any() and not scale[1].any()
    # a code is off by half a step at most, 2^-4 of its value or 2^-10, and the scale and the quotient by 2^-24 each
    size = w.double().abs()
    largest = experts.in_blocks(size).amax((-3, -1))
    step = largest.repeat_interleave(128, -2).repeat_interleave(128, -1)[:, :200, :300]
    off = (experts.values_of(codes, scale) - w.double()).abs()
    assert bool((off <= torch.maximum(2 ** -4 * size, 2 ** -10 / 448 * step) * (1 + 2 ** -10) + 2 ** -22 * size).all())
