"""examples/experts.py on the GPU: layers of experts between allreduces against 64-bit floating point.

Tolerance, derived before the first run, relative to the root mean square of what the layers add.  A rounding to e4m3
is off by at most half a step, which is 1/16 to 1/32 of the value, and evenly within it: 0.045/sqrt(3) = 2.6% in the root
mean square.  Per layer: the norm's codes 2.6%, which the gate and the up projection pass on to their product
(sqrt(2) * 2.6%, the gate's by up to 1.1, silu's largest slope: 4%), the activation's codes 2.6%, the wire's two roundings
3.7% of the summands (FP8; 8-bit integers less), 16-bit roundings below 0.3% each, four of them: 6.1%.  The second layer
passes on the first one's relative error at most three times as large: two layers below 6.1% * (1 + 1 + 3) = 31%.

The router's logits have a standard deviation of 2.  In the first layer each is off by the norm's codes (2.6% of a
normal's deviation: 0.052), the wire's roundings (3.7% of the summands, which are half of the stream's variance: 0.052)
and its rounding to bf16 (2^-9 of at most 8, even: 0.009): 0.074.  Of two logits, and of at most 200 * 64 pairs of a chosen
and another expert, the largest difference's error is below 5 deviations: 5 * sqrt(2) * 0.074 = 0.53."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.parametrize("argv", [
    ["--world", "2", "--tokens", "1", "--hidden", "512", "--inner", "256", "--experts", "8", "--chosen", "2"],
    ["--world", "4", "--tokens", "37", "--hidden", "1032", "--inner", "200", "--experts", "30", "--chosen", "5"],
    ["--world", "8", "--tokens", "200", "--hidden", "1024", "--inner", "72", "--experts", "64", "--chosen", "4", "--codec",
     "Q8"],
    ["--world", "2", "--tokens", "9", "--hidden", "256", "--inner", "136", "--experts", "4", "--chosen", "4"],
])
def test_layers_against_64_bits(argv, capsys):
    assert torch.cuda.is_available()
    import experts
    print(argv, flush=True)
    assert experts.main(argv)[0] < 0.31
    assert "relative error" in capsys.readouterr().out
    error, wrong = experts.main(argv + ["--layers", "1"])
    assert error < 0.10 and wrong < 0.53


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("M", [9, 100])
def test_a_pass_replayed(dtype, M):
    """the same input gives the same bits, whatever the buffers held before: eagerly, in a graph, on another stream, with
    eager work between the replays"""
    import experts
    ex = experts.Experts(4, M, 264, 72, 16, 3, 2, experts.CODECS["Q6"], dtype=dtype, seed=3)
    g = torch.Generator(device="cuda").manual_seed(4)
    h0 = torch.randn(M, 264, generator=g, device="cuda").to(dtype)
    x0 = torch.randn(4, M, 264, generator=g, device="cuda").to(dtype)

    def start():
        ex.h.copy_(h0)
        ex.summands.copy_(x0)

    def result():
        torch.cuda.synchronize()
        return [t.clone() for t in (ex.h, ex.summands, ex.weights, ex.rows, ex.place, *ex.experts)]

    def spoil(fill):
        for t in (ex.gu, ex.out, ex.act_s, ex.s, ex.logits, ex.weights, ex.offsets, ex.rows, ex.place, ex.shared):
            t.fill_(fill)
        ex.q.view(torch.uint8).fill_(fill)

    print("eager", M, dtype, flush=True)
    start()
    ex.run()
    want = result()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        start()
        ex.run()
    for fill in (0, 3, 1):
        print("replay", fill, flush=True)
        spoil(fill)
        graph.replay()
        for a, b in zip(want, result()):
            assert torch.equal(a, b)
        spoil(2)
        start()
        ex.run()                                          # eager work between the replays
        for a, b in zip(want, result()):
            assert torch.equal(a, b)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        start()
        ex.run()
    for a, b in zip(want, result()):
        assert torch.equal(a, b)


def test_two_routes_at_once():
    """on two streams, each with its own workspace"""
    from quantized_two_stage_amd import qr
    T, E, k = 5000, 256, 8
    sets, streams = [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for seed in (1, 2):
        g = torch.Generator(device="cuda").manual_seed(seed)
        i32 = dict(dtype=torch.int32, device="cuda")
        sets.append((torch.randn(T, E, generator=g, device="cuda"), torch.empty(T, k, device="cuda"),
                     torch.empty(T, k, **i32), torch.empty(E + 1, **i32), torch.empty(T * k, **i32),
                     torch.empty(T, k, **i32), qr.alloc_route_workspace(T, E, k)))
    want = []
    for s in sets:
        qr.qr_route(*s[:6], workspace=s[6])
        torch.cuda.synchronize()
        want.append([t.clone() for t in s[1:6]])
    for _ in range(20):
        for s, stream in zip(sets, streams):
            qr.qr_route(*s[:6], workspace=s[6], stream=stream)
    torch.cuda.synchronize()
    for s, w in zip(sets, want):
        assert all(torch.equal(a, b) for a, b in zip(s[1:6], w))
