"""Feed-forward layers with a mixture of experts in 8-bit floating point: the operators of include/qr_f8.h between two
allreduces, as a serving program calls them.  The ranks are simulated on one GPU, as everywhere in this library.

A layer, on every rank:

    the allreduce of the last layer's outputs                          qr_quantize_recv, qr_reduce_recv, qr_gather_stage2
    its values + residual, normalised, in 8-bit codes                  qr_add_rmsnorm_f8
    the router's logits; every token's experts and their rows          qr_gemm_f8, qr_route
    the experts' gate and up projections, on the tokens' codes in place    qr_gemm_f8_grouped
    silu(gate) * up, in 8-bit codes                                    qr_silu_mul_f8
    the experts' down projections (this rank's inner channels)         qr_gemm_f8_grouped
    a shared expert, on every token                                    qr_gemm_f8, qr_silu_mul_f8, qr_gemm_f8
    the weighted sum: this rank's summand of the layer's output        qr_combine

A pass is captured into a HIP graph and replayed; the result is compared with the same layers in 64-bit floating point,
with the experts that the router chose.

    python examples/experts.py [--world 8] [--tokens 16] [--hidden 4096] [--inner 256] [--experts 32] [--chosen 4]
                               [--layers 2] [--codec FP8]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from quantized_two_stage_amd import qr  # noqa: E402

CODECS = {"FP": qr.QR_FP, "FP8": qr.QR_FP8, "Q8": qr.QR_Q8, "Q6": qr.QR_Q6, "Q4": qr.QR_Q4}
EPS = 1e-5


def blocks(n):
    return -(-n // 128)


def in_blocks(w):
    """[..., N, K] filled up to whole blocks, as [..., N blocks, 128, K blocks, 128]."""
    N, K = w.shape[-2:]
    full = w.new_zeros(*w.shape[:-2], blocks(N) * 128, blocks(K) * 128)
    full[..., :N, :K] = w
    return full.unflatten(-2, (-1, 128)).unflatten(-1, (-1, 128))


def codes_of(w):
    """Weights [..., N, K] as e4m3 codes with a scale for each block of 128 x 128."""
    N, K = w.shape[-2:]
    b = in_blocks(w)
    scale = b.abs().amax((-3, -1)) / 448
    codes = torch.empty(*w.shape[:-1], -(-K // 16) * 16, dtype=torch.float8_e4m3fn, device=w.device)[..., :K]
    divisor = torch.where(scale > 0, scale, 1.0)             # a block of zeros has codes 0 and scale 0
    codes.copy_((b / divisor[..., :, None, :, None]).flatten(-2).flatten(-3, -2)[..., :N, :K])
    return codes, scale


def values_of(codes, scale):
    """The weights that codes stand for, in 64 bits."""
    return (in_blocks(codes.double()) * scale.double()[..., :, None, :, None]).flatten(-2).flatten(
        -3, -2)[..., :codes.shape[-2], :codes.shape[-1]]


class Experts:
    """The layers' weights and the buffers of a pass: W ranks, M tokens, hidden size d, f inner channels of an expert a
    rank, E experts, k of them for a token."""

    def __init__(self, W, M, d, f, E, k, layers, codec, dtype=torch.bfloat16, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)

        def randn(*size):
            return torch.randn(*size, generator=g, device=device)

        self.W, self.M, self.d, self.f, self.E, self.k, self.codec = W, M, d, f, E, k, codec
        self.wire_dtype = qr.QR_FP16 if dtype is torch.float16 else qr.QR_BF16
        # per layer: the norm's weight, the router and, per rank, the experts' and the shared expert's two products
        self.layers = [dict(norm=(1 + 0.1 * randn(d)).to(dtype), router=codes_of(randn(E, d) * (2 / d ** 0.5)),
                            first=[codes_of(randn(E, 2 * f, d) / d ** 0.5) for _ in range(W)],
                            second=[codes_of(randn(E, d, f) / (W * f) ** 0.5) for _ in range(W)],
                            shared1=[codes_of(randn(2 * f, d) / d ** 0.5) for _ in range(W)],
                            shared2=[codes_of(randn(d, f) / (W * f) ** 0.5) for _ in range(W)])
                       for _ in range(layers)]
        n = M * d

        def empty(*size):
            return torch.empty(*size, dtype=dtype, device=device)

        def i32(*size):
            return torch.empty(*size, dtype=torch.int32, device=device)

        self.summands, self.x = empty(W, M, d), empty(M, d)
        self.recv, self.reduced = qr.alloc_recv(W, codec, n, device), qr.alloc_wire(codec, n, device)
        self.h = empty(M, d)
        self.q, self.s = qr.alloc_f8(M, d, device)
        self.logits = empty(M, E)
        self.weights = torch.empty(M, k, device=device)
        self.experts = [i32(M, k) for _ in range(layers)]        # kept apart for the comparison
        self.offsets, self.rows, self.place = i32(E + 1), i32(M * k), i32(M, k)
        self.ws = qr.alloc_route_workspace(M, E, k, device)
        self.gu, self.out = empty(M * k, 2 * f), empty(M * k, d)
        self.act, self.act_s = qr.alloc_f8(M * k, f, device)
        self.shared = empty(M, d)

    def _allreduce(self):
        qr.qr_quantize_recv(self.codec, list(self.summands), self.recv)
        qr.qr_reduce_recv(self.codec, self.W, self.recv, self.M * self.d, self.reduced, self.wire_dtype)
        qr.qr_gather_stage2(self.codec, self.reduced, [self.x])

    def run(self):
        """The residual stream h and the ranks' summands of the first layer's input, in place, to those after the last
        layer; returns h, with the last layer's output still to be added, and that output's summands."""
        M, gu, act, act_s = self.M, self.gu, self.act, self.act_s
        for p, experts in zip(self.layers, self.experts):
            self._allreduce()
            qr.qr_add_rmsnorm_f8(self.x, self.h, p["norm"], EPS, self.h, None, self.q, self.s)
            qr.qr_gemm_f8(self.q, self.s, *p["router"], self.logits)
            qr.qr_route(self.logits, self.weights, experts, self.offsets, self.rows, self.place, renormalize=True,
                        workspace=self.ws)
            for r in range(self.W):                       # on a node: every rank its own
                qr.qr_gemm_f8(self.q, self.s, *p["shared1"][r], gu[:M])
                qr.qr_silu_mul_f8(gu[:M], act[:M], act_s[:M])
                qr.qr_gemm_f8(act[:M], act_s[:M], *p["shared2"][r], self.shared)
                qr.qr_gemm_f8_grouped(self.q, self.s, *p["first"][r], self.offsets, gu, rows=self.rows)
                qr.qr_silu_mul_f8(gu, act, act_s)
                qr.qr_gemm_f8_grouped(act, act_s, *p["second"][r], self.offsets, self.out)
                qr.qr_combine(self.out, self.place, self.weights, self.summands[r], addend=self.shared)
        return self.h, self.summands

    def reference(self, h, summands):
        """The residual stream after the last layer in 64 bits, nothing rounded but the weights' codes; the experts are
        those of the last pass.  Also how far, at most, an expert that was not chosen lies above one that was."""
        h, x = h.double(), summands.double().sum(0)
        wrong = 0.0
        for p, experts in zip(self.layers, self.experts):
            h = h + x
            u = h * (h.square().mean(1, keepdim=True) + EPS).rsqrt() * p["norm"].double()
            logits = u @ values_of(*p["router"]).t()
            chosen = logits.gather(1, experts.long())
            if self.k < self.E:
                others = logits.scatter(1, experts.long(), -torch.inf).amax(1)
                wrong = max(wrong, float((others - chosen.amin(1)).max()))
            weight = torch.softmax(chosen, 1)
            x = torch.zeros_like(h)

            def forward(u, w1, w2):
                gate, up = (u @ w1.t()).split(self.f, 1)
                return (gate * torch.sigmoid(gate) * up) @ w2.t()

            for r in range(self.W):
                x += forward(u, values_of(*p["shared1"][r]), values_of(*p["shared2"][r]))
                w1, w2 = values_of(*p["first"][r]), values_of(*p["second"][r])
                for e in range(self.E):
                    token, slot = (experts == e).nonzero(as_tuple=True)
                    if token.numel():
                        x.index_add_(0, token, weight[token, slot][:, None] * forward(u[token], w1[e], w2[e]))
        return h + x, wrong


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--world", type=int, default=8, choices=[2, 4, 8])
    p.add_argument("--tokens", type=int, default=16)
    p.add_argument("--hidden", type=int, default=4096)
    p.add_argument("--inner", type=int, default=256, help="inner channels of an expert on one rank")
    p.add_argument("--experts", type=int, default=32)
    p.add_argument("--chosen", type=int, default=4, help="experts of a token")
    p.add_argument("--layers", type=int, default=2)
    p.add_argument("--codec", default="FP8", choices=sorted(CODECS))
    a = p.parse_args(argv)
    ex = Experts(a.world, a.tokens, a.hidden, a.inner, a.experts, a.chosen, a.layers, CODECS[a.codec])
    g = torch.Generator(device="cuda").manual_seed(1)
    h0 = torch.randn(a.tokens, a.hidden, generator=g, device="cuda").to(ex.h.dtype)
    x0 = (torch.randn(ex.summands.shape, generator=g, device="cuda") / a.world ** 0.5).to(ex.h.dtype)

    def start():
        ex.h.copy_(h0)
        ex.summands.copy_(x0)

    start()
    ex.run()                                              # loads the kernels before the capture
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        start()
        ex.run()
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    graph.replay()
    begin.record()
    for _ in range(10):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    want, wrong = ex.reference(h0, x0)
    got = ex.h.double() + ex.summands.double().sum(0)
    # against what the layers add to the residual stream
    error = float((got - want).norm() / (want - h0.double()).norm())
    print("%d layers, %d ranks, %d tokens, hidden %d, %d experts of %d inner channels a rank, %d a token, %s on the "
          "wire: %.1f us a pass of all ranks, relative error %.4f, router off by %.3f"
          % (a.layers, a.world, a.tokens, a.hidden, a.experts, a.inner, a.chosen, a.codec,
             begin.elapsed_time(end) * 100, error, wrong))
    return error, wrong


if __name__ == "__main__":
    main()
