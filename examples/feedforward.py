"""Feed-forward layers of a tensor-parallel transformer in 8-bit integers: the operators of include/qr_layer.h between
two allreduces, as a serving program calls them.  The ranks are simulated on one GPU, as everywhere in this library.

A layer, on every rank:

    the allreduce of the last layer's outputs, up to its reduced wire image    qr_quantize_recv, qr_reduce_recv
    its values + residual, normalised, in 8-bit codes                          qr_gather_add_rmsnorm_q8
    gate and up projection (this rank's columns)                               qr_gemm_i8
    silu(gate) * up, in 8-bit codes                                            qr_silu_mul_q8
    down projection (this rank's rows): its summand of the layer's output      qr_gemm_i8

The allreduce's values are never written: the norm reads them from the wire.  A pass is captured into a HIP graph and
replayed; the result is compared with the same layers in 64-bit floating point.

    python examples/feedforward.py [--world 8] [--tokens 16] [--hidden 8192] [--inner 4096] [--layers 2] [--codec Q8]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from quantized_two_stage_amd import qr  # noqa: E402

CODECS = {"FP": qr.QR_FP, "Q8": qr.QR_Q8, "Q6": qr.QR_Q6, "Q4": qr.QR_Q4, "FP8": qr.QR_FP8}
EPS = 1e-5


def codes_of(w):
    """Weights [N, K] as 8-bit codes with a scale for each output channel."""
    scale = w.abs().amax(1) / 127
    codes, _ = qr.alloc_q8(*w.shape, device=w.device)
    codes.copy_((w / scale[:, None]).round_())
    return codes, scale


class FeedForward:
    """The layers' weights and the buffers of a pass: W ranks, M tokens, hidden size d, f inner channels a rank."""

    def __init__(self, W, M, d, f, layers, codec, dtype=torch.bfloat16, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)

        def randn(*size):
            return torch.randn(*size, generator=g, device=device)

        self.W, self.M, self.d, self.f, self.codec = W, M, d, f, codec
        self.wire_dtype = qr.QR_FP16 if dtype is torch.float16 else qr.QR_BF16
        # per layer: the norm's weight and, per rank, codes and scales of both products
        self.layers = [((1 + 0.1 * randn(d)).to(dtype),
                        [codes_of(randn(2 * f, d) / d ** 0.5) for _ in range(W)],
                        [codes_of(randn(d, f) / (W * f) ** 0.5) for _ in range(W)]) for _ in range(layers)]
        self.last = (1 + 0.1 * randn(d)).to(dtype)
        n = M * d
        self.summands = torch.empty(W, M, d, dtype=dtype, device=device)
        self.recv, self.reduced = qr.alloc_recv(W, codec, n, device), qr.alloc_wire(codec, n, device)
        self.h = torch.empty(M, d, dtype=dtype, device=device)
        self.q, self.s = qr.alloc_q8(M, d, device)
        self.gu = torch.empty(M, 2 * f, dtype=dtype, device=device)
        self.act, self.act_s = qr.alloc_q8(M, f, device)

    def _reduce_and_norm(self, weight):
        qr.qr_quantize_recv(self.codec, list(self.summands), self.recv)
        qr.qr_reduce_recv(self.codec, self.W, self.recv, self.M * self.d, self.reduced, self.wire_dtype)
        qr.qr_gather_add_rmsnorm_q8(self.codec, self.reduced, self.h, weight, EPS, self.h, self.q, self.s)

    def run(self):
        """The residual stream h and the ranks' summands of the first layer's input, in place, to those after the
        last layer; returns h and the codes and scales of its norm."""
        for weight, first, second in self.layers:
            self._reduce_and_norm(weight)
            for r in range(self.W):                       # on a node: every rank its own
                qr.qr_gemm_i8(self.q, self.s, *first[r], self.gu)
                qr.qr_silu_mul_q8(self.gu, self.act, self.act_s)
                qr.qr_gemm_i8(self.act, self.act_s, *second[r], self.summands[r])
        self._reduce_and_norm(self.last)
        return self.h, self.q, self.s

    def reference(self, h, summands):
        """The residual stream after the last layer in 64 bits, nothing rounded but the weights' codes."""
        h, x = h.double(), summands.double().sum(0)
        for weight, first, second in self.layers:
            h = h + x
            u = h * (h.square().mean(1, keepdim=True) + EPS).rsqrt() * weight.double()
            x = torch.zeros_like(h)
            for (b1, s1), (b2, s2) in zip(first, second):
                gate, up = ((u @ b1.double().t()) * s1.double()).split(self.f, 1)
                x += ((gate * torch.sigmoid(gate) * up) @ b2.double().t()) * s2.double()
        return h + x


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--world", type=int, default=8, choices=[2, 4, 8])
    p.add_argument("--tokens", type=int, default=16)
    p.add_argument("--hidden", type=int, default=8192)
    p.add_argument("--inner", type=int, default=4096, help="inner channels of one rank")
    p.add_argument("--layers", type=int, default=2)
    p.add_argument("--codec", default="Q8", choices=sorted(CODECS))
    a = p.parse_args(argv)
    ff = FeedForward(a.world, a.tokens, a.hidden, a.inner, a.layers, CODECS[a.codec])
    g = torch.Generator(device="cuda").manual_seed(1)
    h0 = torch.randn(a.tokens, a.hidden, generator=g, device="cuda").to(ff.h.dtype)
    x0 = (torch.randn(ff.summands.shape, generator=g, device="cuda") / a.world ** 0.5).to(ff.h.dtype)
    want = ff.reference(h0, x0)

    def start():
        ff.h.copy_(h0)
        ff.summands.copy_(x0)

    start()
    ff.run()                                              # loads the kernels before the capture
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        start()
        ff.run()
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    graph.replay()
    begin.record()
    for _ in range(10):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    # against what the layers add to the residual stream
    error = float((ff.h.double() - want).norm() / (want - h0.double()).norm())
    print("%d layers, %d ranks, %d tokens, hidden %d, inner %d a rank, %s on the wire: %.1f us a pass of all ranks, "
          "relative error %.4f" % (a.layers, a.world, a.tokens, a.hidden, a.inner, a.codec,
                                   begin.elapsed_time(end) * 100, error))
    return error


if __name__ == "__main__":
    main()
