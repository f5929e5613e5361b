"""The operators of a tensor-parallel layer between two allreduces, as workloads to measure.

Four operators, in the order a layer runs them:

- ``wire``: the reduced wire image of an allreduce is dequantized, the residual is added, the sum is normalised by
  its root mean square and leaves in 8-bit codes with one scale a token;
- ``norm``: the same from a 16-bit buffer;
- ``gemm``: the product of 8-bit codes, with a scale for each token and each output channel;
- ``act``: silu(gate) * up of the first product's output, in 8-bit codes with one scale a token.

``run`` computes them in elementary torch operations, or, where ``own`` is true, with the library's kernels.  Codes
are returned as the 16-bit values they stand for.
"""
import math

import torch

own = False

FP, Q8, Q6, Q4, FP8, Q8A, Q6A, Q4A = 0, 1, 2, 3, 5, 9, 10, 11
BITS = {FP: 16, Q8: 8, Q6: 6, Q4: 4, FP8: 8, Q8A: 8, Q6A: 6, Q4A: 4}
TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}
EPS = 1e-5
TINY = 2.0 ** -119          # a row whose largest magnitude is below this counts as zero
DEVICE = "cuda"


def listed():
    return [
        # the norm before a layer for one token of one sequence: latency counts, not bandwidth
        dict(name="norm_token", op="norm", dtype="bf16", M=1, d=8192, pad=0),
        # a prefill's remainder with an odd width: no row after the first starts at a 16-byte boundary
        dict(name="norm_ragged", op="norm", dtype="fp16", M=333, d=5003, pad=0),
        # a long prefill
        dict(name="norm_prefill", op="norm", dtype="bf16", M=8192, d=8192, pad=0),
        # sixteen sequences decoding, the allreduce's result in 8-bit wire codes
        dict(name="wire_batch", op="wire", dtype="fp16", M=16, d=8192, codec=Q8),
        # 1024 tokens of hidden size 8192 in 6-bit wire codes, the allreduce workload of that shape
        dict(name="wire_tokens", op="wire", dtype="bf16", M=1024, d=8192, codec=Q6),
        # 64 MB of 16-bit values a rank, asymmetric 4-bit wire codes: the largest allreduce workload
        dict(name="wire_prefill", op="wire", dtype="fp16", M=4096, d=8192, codec=Q4A),
        # eight sequences decoding: one rank's share of the gated activation
        dict(name="act_batch", op="act", dtype="bf16", M=8, d=4096),
        # the same share for a long prefill
        dict(name="act_prefill", op="act", dtype="bf16", M=8192, d=4096),
        # one token through one rank's first product: the weights' bytes bound it
        dict(name="gemm_token", op="gemm", dtype="bf16", M=1, N=8192, K=8192, bias=False),
        # a decoding batch through one rank's second product, with a bias
        dict(name="gemm_batch", op="gemm", dtype="fp16", M=48, N=8192, K=4096, bias=True),
        # sizes that no tile divides
        dict(name="gemm_ragged", op="gemm", dtype="bf16", M=333, N=5003, K=2050, bias=False),
        # a long prefill: the matrix units' rate bounds it
        dict(name="gemm_prefill", op="gemm", dtype="bf16", M=8192, N=8192, K=8192, bias=False),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "wire", "act", "gemm", "gemm"])
    dtype = rng.choice(["bf16", "fp16"])
    if op == "gemm":
        K = _log_int(rng, 64, 16384)
        if rng.random() < 0.5:
            K = max(64, K // 64 * 64)
        N = _log_int(rng, 64, 16384)
        if rng.random() < 0.5:
            N = max(64, N // 64 * 64)
        M = _log_int(rng, 1, max(1, min(8192, 8192 ** 3 // (N * K))))
        return dict(op=op, dtype=dtype, M=M, N=N, K=K, bias=rng.random() < 0.5)
    d = _log_int(rng, 64, 16384)
    if op == "wire" or rng.random() < 0.7:
        d = d // 8 * 8
    if op == "act":
        return dict(op=op, dtype=dtype, M=_log_int(rng, 1, min(8192, 2 ** 25 // d)), d=d)
    if op == "wire":
        return dict(op=op, dtype=dtype, M=_log_int(rng, 1, min(8192, 2 ** 25 // d)), d=d,
                    codec=rng.choice([FP, Q8, Q6, Q4, FP8, Q8A, Q6A, Q4A]))
    return dict(op=op, dtype=dtype, M=_log_int(rng, 1, min(8192, 2 ** 26 // d)), d=d, pad=rng.choice([0, 0, 8, 3]))


def _wire_planes(codec, n):
    """(bytes of codes, offset of the scales, offset of the zeros or None, bytes in all) of a wire image."""
    if codec == FP:
        return 2 * n, None, None, 2 * n
    nb = -(-n // 32)
    codes = nb * 4 * BITS[codec]
    at_s = -(-codes // 256) * 256
    end = at_s + 2 * nb
    if codec < 8:
        return codes, at_s, None, end
    at_z = -(-end // 256) * 256
    return codes, at_s, at_z, at_z + 2 * nb


def _make_wire(codec, n, dtype, g):
    """A wire image of n activations of about unit variance: blocks of 32 with a binary16 scale (and zero)."""
    codes_bytes, at_s, at_z, total = _wire_planes(codec, n)
    if codec == FP:
        return torch.randn(n, generator=g, device=DEVICE).to(dtype).view(torch.uint8)
    wire = torch.zeros(total, dtype=torch.uint8, device=DEVICE)
    nb, b = -(-n // 32), BITS[codec]
    size = torch.rand(nb, 1, generator=g, device=DEVICE) * 2 + 1.5           # the block's largest magnitude
    t = (torch.randn(nb, 32, generator=g, device=DEVICE) / 2.2).clamp_(-1, 1)
    if codec == FP8:
        code = (t * 448).to(torch.float8_e4m3fn).view(torch.uint8)
        scale = size / 448
    elif at_z is None:
        top = 2 ** (b - 1) - 1
        code = (t * top).round().to(torch.int16) & (2 ** b - 1)
        scale = size / top
    else:
        top = 2 ** b - 1
        code = ((t + 1) * (top / 2)).round().to(torch.int16)
        scale = 2 * size / top
        wire[at_z:at_z + 2 * nb] = (-size + 0.1).to(torch.float16).view(torch.uint8).reshape(-1)
    if b == 6:
        c = code.reshape(-1, 4)
        packed = torch.stack([(c[:, 0] | (c[:, 1] << 6)) & 255, ((c[:, 1] >> 2) | (c[:, 2] << 4)) & 255,
                              ((c[:, 2] >> 4) | (c[:, 3] << 2)) & 255], 1)
    elif b == 4:
        c = code.reshape(-1, 2)
        packed = c[:, 0] | (c[:, 1] << 4)
    else:
        packed = code
    wire[:codes_bytes] = packed.to(torch.uint8).reshape(-1)
    wire[at_s:at_s + 2 * nb] = scale.to(torch.float16).view(torch.uint8).reshape(-1)
    return wire


def _unpack(codec, wire, n, dtype, real):
    """The n values that a wire image holds, in the type `real`, rounded to the buffer type."""
    codes_bytes, at_s, at_z, _ = _wire_planes(codec, n)
    if codec == FP:
        return wire.view(dtype).to(real)
    nb, b = -(-n // 32), BITS[codec]
    raw = wire[:codes_bytes]
    if codec == FP8:
        c = raw.view(torch.float8_e4m3fn).to(real)
    elif b == 8:
        c = (raw if at_z is not None else raw.view(torch.int8)).to(real)
    else:
        if b == 4:
            c = torch.stack([raw & 15, raw >> 4], 1)
        else:
            q = raw.reshape(-1, 3).to(torch.int16)
            c = torch.stack([q[:, 0] & 63, (q[:, 0] >> 6) | ((q[:, 1] & 15) << 2),
                             (q[:, 1] >> 4) | ((q[:, 2] & 3) << 4), q[:, 2] >> 2], 1)
        c = c.to(real)
        if at_z is None:
            c = torch.where(c >= 2 ** (b - 1), c - 2 ** b, c)
    v = c.reshape(nb, 32) * wire[at_s:at_s + 2 * nb].view(torch.float16).to(real)[:, None]
    if at_z is not None:
        v = v + wire[at_z:at_z + 2 * nb].view(torch.float16).to(real)[:, None]
    return v.reshape(-1)[:n].to(dtype).to(real)


def _codes_like(M, d):
    """An [M, d] buffer of 8-bit codes whose rows start at 16-byte boundaries."""
    return torch.zeros(M, -(-d // 16) * 16, dtype=torch.int8, device=DEVICE)[:, :d]


def prepare(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)
    dtype, M = TYPES[case["dtype"]], case["M"]
    randn = lambda *size: torch.randn(*size, generator=g, device=DEVICE)  # noqa: E731
    s = dict(case, dtype=dtype)
    if case["op"] == "gemm":
        N, K = case["N"], case["K"]
        s["a"], s["b"] = _codes_like(M, K), _codes_like(N, K)
        for t in (s["a"], s["b"]):
            # codes of rows whose largest magnitude is 3 to 5 standard deviations
            t.copy_((randn(t.shape) * (25 + 17 * torch.rand(t.shape[0], 1, generator=g, device=DEVICE))).round_()
                    .clamp_(-127, 127))
        s["sa"] = (torch.rand(M, generator=g, device=DEVICE) + 0.5) * 0.03
        s["sb"] = (torch.rand(N, generator=g, device=DEVICE) + 0.5) * (0.03 / math.sqrt(K))
        s["bias"] = (randn(N) * 0.5).to(dtype) if case["bias"] else None
        s["c"] = torch.empty(M, N, dtype=dtype, device=DEVICE)
        return s
    d = case["d"]
    s["q"] = _codes_like(M, d)
    s["scales"] = torch.empty(M, 1, dtype=torch.float32, device=DEVICE)
    s["values"] = torch.empty(M, d, dtype=dtype, device=DEVICE)
    if case["op"] == "act":
        s["gu"] = (randn(M, 2 * d) * 1.5).to(dtype)
        return s
    # a residual stream: larger than a layer's output, with a few channels larger still
    channel = torch.where(torch.rand(d, generator=g, device=DEVICE) < 0.002, 20.0, 1.0)
    s["residual"] = (randn(M, d).mul_(3.0).mul_(channel)).to(dtype)
    s["weight"] = (1 + 0.2 * randn(d)).to(dtype)
    s["h"] = torch.empty(M, d, dtype=dtype, device=DEVICE)
    if case["op"] == "wire":
        s["wire"] = _make_wire(case["codec"], M * d, dtype, g)
    else:
        s["x"] = randn(M, d + case["pad"]).to(dtype)[:, :d]
    return s


def _codes(u, factor):
    """Codes of the rows of u (their largest magnitude is 127 steps), as the values they stand for where u is times
    `factor`, and their scales."""
    a = u.abs().amax(1, keepdim=True)
    fine = torch.isfinite(a) & torch.isfinite(factor)
    use = fine & (a >= TINY)
    code = torch.where(use, torch.round(u * (127.0 / torch.where(use, a, 1.0))), 0.0)
    scale = torch.where(fine, torch.where(use, a * factor / 127.0, 0.0), math.nan)
    return code * scale, scale


def _norm(x, residual, weight, dtype, real):
    h = (x.to(real) + residual.to(real)).to(dtype)
    hr = h.to(real)
    factor = torch.rsqrt((hr * hr).sum(1, keepdim=True) / hr.shape[1] + EPS)
    values, scale = _codes(hr * weight.to(real), factor)
    return h, values, scale


def _act(gu, d, real):
    g, u = gu[:, :d].to(real), gu[:, d:].to(real)
    v = g / (1 + torch.exp(-g)) * u
    return _codes(v, torch.ones_like(v[:, :1]))


def _gemm(s, real):
    acc = torch.matmul(s["a"].to(real), s["b"].to(real).t())
    c = acc * s["sa"].to(real)[:, None] * s["sb"].to(real)[None, :]
    return c if s["bias"] is None else c + s["bias"].to(real)


def _run_own(s):
    from quantized_two_stage_amd import qr
    if s["op"] == "gemm":
        if "workspace" not in s:        # kept with the layer, as its weights are
            s["workspace"] = qr.alloc_gemm_workspace(s["M"], s["N"], s["K"])
        qr.qr_gemm_i8(s["a"], s["sa"], s["b"], s["sb"], s["c"], bias=s["bias"], workspace=s["workspace"])
        return {"c": s["c"]}
    if s["op"] == "act":
        qr.qr_silu_mul_q8(s["gu"], s["q"], s["scales"])
        out = {}
    elif s["op"] == "wire":
        qr.qr_gather_add_rmsnorm_q8(s["codec"], s["wire"], s["residual"], s["weight"], EPS, s["h"], s["q"],
                                    s["scales"])
        out = {"h": s["h"]}
    else:
        qr.qr_add_rmsnorm_q8(s["x"], s["residual"], s["weight"], EPS, s["h"], s["q"], s["scales"])
        out = {"h": s["h"]}
    torch.mul(s["q"], s["scales"], out=s["values"])
    return dict(out, values=s["values"], scales=s["scales"])


def run(s):
    if own:
        return _run_own(s)
    real = torch.float32
    if s["op"] == "gemm":
        return {"c": _gemm(s, real).to(s["dtype"])}
    if s["op"] == "act":
        values, scale = _act(s["gu"], s["d"], real)
        return {"values": values.to(s["dtype"]), "scales": scale}
    if s["op"] == "wire":
        x = _unpack(s["codec"], s["wire"], s["M"] * s["d"], s["dtype"], real).reshape(s["M"], s["d"])
    else:
        x = s["x"]
    h, values, scale = _norm(x, s["residual"], s["weight"], s["dtype"], real)
    return {"h": h, "values": values.to(s["dtype"]), "scales": scale}


def exact(case, seed):
    """The same from the definition in 64 bits; nothing is rounded but what the definition rounds (the sum with the
    residual, a wire value, the codes)."""
    s = prepare(case, seed)
    f64 = torch.float64
    if s["op"] == "gemm":
        c = torch.empty(s["M"], s["N"], dtype=f64, device=DEVICE)
        b = s["b"].to(f64).t()
        for i in range(0, s["M"], 2048):
            c[i:i + 2048] = s["a"][i:i + 2048].to(f64) @ b
        c *= s["sa"].to(f64).unsqueeze(1) * s["sb"].to(f64)
        if s["bias"] is not None:
            c += s["bias"].to(f64)
        return {"c": c}
    M, d = s["M"], s["d"]
    out = {}
    if s["op"] == "act":
        gate, up = s["gu"].to(f64).split(d, dim=1)
        v = gate * torch.sigmoid(gate) * up
        gain = torch.ones(M, 1, dtype=f64, device=DEVICE)
    else:
        if s["op"] == "wire":
            x = _unpack(s["codec"], s["wire"], M * d, s["dtype"], f64).reshape(M, d)
        else:
            x = s["x"].to(f64)
        out["h"] = (x + s["residual"].to(f64)).to(s["dtype"]).to(f64)
        gain = out["h"].square().mean(1, keepdim=True).add(EPS).pow(-0.5)
        v = out["h"] * s["weight"].to(f64)
    step = v.abs().amax(1, keepdim=True) / 127
    out["values"] = torch.where(step > 0, torch.round(v / step), 0.0) * step * gain
    out["scales"] = step * gain
    return out


def work(case):
    M = case["M"]
    if case["op"] == "gemm":
        N, K = case["N"], case["K"]
        return {"bytes": M * K + N * K + 2 * M * N + 4 * (M + N) + (2 * N if case["bias"] else 0),
                "flops": 2 * M * N * K}
    d = case["d"]
    if case["op"] == "act":
        return {"bytes": M * d * (4 + 1) + 4 * M, "flops": 10 * M * d}
    read = _wire_planes(case["codec"], M * d)[3] if case["op"] == "wire" else 2 * M * d
    return {"bytes": read + M * d * (2 + 2 + 1) + 2 * d + 4 * M, "flops": 8 * M * d}
