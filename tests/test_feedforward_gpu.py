"""examples/feedforward.py on the GPU: two feed-forward layers between allreduces against 64-bit floating point.

Tolerance, derived before the first run, relative to the root mean square of what the layers add.  A rounding to steps
of max/127 is off by max/(127 sqrt(12)) in the root mean square: with max at most 5 standard deviations of a row of
normals, 1.2% for the norm's codes; with max at most 12 of silu(gate)*up (a product of two normals and a gate), 2.8% for
the activation's; with max at most 3 of a block of 32, 0.7% for each of the wire's two 8-bit roundings, three times.  16-bit
roundings are below 0.3% each.  The second layer passes on the first one's relative error at most three times as large
(its derivative: the gate's and the up projection's, each of a norm).  Independent errors add in quadrature:
per layer sqrt(1.2^2 + 2.8^2 + 2 * 0.7^2 + 4 * 0.3^2) = 3.3%; two layers, the first carried by 1 + 3, below 14%."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.parametrize("argv", [
    ["--world", "2", "--tokens", "1", "--hidden", "512", "--inner", "384"],
    ["--world", "4", "--tokens", "37", "--hidden", "1032", "--inner", "200"],
    ["--world", "8", "--tokens", "130", "--hidden", "1024", "--inner", "136", "--codec", "FP"],
])
def test_layers_against_64_bits(argv, capsys):
    assert torch.cuda.is_available()
    import feedforward
    print(argv, flush=True)
    assert feedforward.main(argv) < 0.14
    assert "relative error" in capsys.readouterr().out


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_a_pass_can_be_repeated(dtype):
    """the same input gives the same bits, whatever the buffers held before"""
    import feedforward
    ff = feedforward.FeedForward(4, 9, 264, 72, 2, feedforward.CODECS["Q6"], dtype=dtype, seed=3)
    g = torch.Generator(device="cuda").manual_seed(4)
    h0 = torch.randn(9, 264, generator=g, device="cuda").to(dtype)
    x0 = torch.randn(4, 9, 264, generator=g, device="cuda").to(dtype)
    outs = []
    for fill in (0, 3):
        for buf in (ff.gu, ff.act, ff.act_s, ff.q, ff.s):
            buf.fill_(fill)
        ff.h.copy_(h0)
        ff.summands.copy_(x0)
        outs.append([t.clone() for t in ff.run()])
    torch.cuda.synchronize()
    for a, b in zip(*outs):
        assert torch.equal(a, b)
