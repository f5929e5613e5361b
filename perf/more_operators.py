"""The operators in 8-bit floating point between two allreduces, dense and by experts, as workloads to measure.

- ``norm``: residual addition and root-mean-square norm to e4m3 codes with a scale for each block of 128 channels, and
  the normed values in 16 bits, which a router reads;
- ``act``: silu(gate) * up to such codes;
- ``gemm``: the product of such codes, the weights with a scale for each block of 128 x 128;
- ``grouped``: the same with the tokens' rows grouped by expert, each group with its own weights;
- ``route``: every token's k experts, their weights, and the rows in the experts' order;
- ``combine``: the weighted sum of a token's k rows.

``run`` computes them in elementary torch operations, or, where ``own`` is true, with the library's kernels.  Codes
are returned as the values they stand for.
"""
import math

import torch

own = False

TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
F8 = torch.float8_e4m3fn
BLOCK = 128
EPS = 1e-5
TINY = 2.0 ** -119          # a block whose largest magnitude is below this counts as zero
DEVICE = "cuda"


def listed():
    return [
        # the norm before a router for one token of one sequence: latency counts, not bandwidth
        dict(name="norm_token", op="norm", dtype="bf16", M=1, d=8192, y=True),
        # a prefill of an odd width, no router behind it: no row after the first starts at a 16-byte boundary
        dict(name="norm_ragged", op="norm", dtype="fp16", M=3000, d=5003, y=False),
        # a few rows of an inner size that no block divides
        dict(name="act_ragged", op="act", dtype="fp16", M=333, d=1000),
        # the rows of a prefill of 4096 tokens, eight experts a token
        dict(name="act_prefill", op="act", dtype="bf16", M=32768, d=1024),
        # one token through one rank's first product: the weights' bytes bound it
        dict(name="gemm_token", op="gemm", dtype="bf16", M=1, N=8192, K=8192, bias=False),
        # a long prefill: the matrix units' rate bounds it
        dict(name="gemm_prefill", op="gemm", dtype="bf16", M=8192, N=8192, K=8192, bias=True),
        # sixteen sequences decoding: the first product of four experts a token, tokens read where they lie
        dict(name="grouped_batch", op="grouped", dtype="fp16", T=16, k=4, E=32, N=2048, K=8192, gather=True, bias=False),
        # the second product of a long prefill over many experts
        dict(name="grouped_prefill", op="grouped", dtype="bf16", T=4096, k=8, E=64, N=8192, K=1024, gather=False,
             bias=False),
        # a decoding batch's router
        dict(name="route_batch", op="route", dtype="fp32", T=16, k=4, E=32, renormalize=True),
        # a long prefill's router
        dict(name="route_prefill", op="route", dtype="bf16", T=16384, k=8, E=256, renormalize=False),
        # a decoding batch of an odd width, beside a shared expert's output
        dict(name="combine_ragged", op="combine", dtype="fp16", T=17, k=4, d=5003, addend=True),
        # a long prefill
        dict(name="combine_prefill", op="combine", dtype="bf16", T=4096, k=8, d=8192, addend=False),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _size(rng, lo, hi):
    """A row length: half of them multiples of the block."""
    n = _log_int(rng, lo, hi)
    return max(BLOCK, n // BLOCK * BLOCK) if rng.random() < 0.5 else n


def draw(rng):
    op = rng.choice(["norm", "act", "gemm", "gemm", "grouped", "grouped", "route", "combine"])
    dtype = rng.choice(["bf16", "fp16"])
    if op == "gemm":
        K, N = _size(rng, 64, 16384), _size(rng, 64, 16384)
        M = _log_int(rng, 1, max(1, min(8192, 8192 ** 3 // (N * K))))
        return dict(op=op, dtype=dtype, M=M, N=N, K=K, bias=rng.random() < 0.5)
    if op in ("grouped", "route", "combine"):
        E = _log_int(rng, 4, 128 if op == "grouped" else 512)
        k = rng.randint(1, min(8, E))
    if op == "grouped":
        K = _size(rng, 64, 8192)
        N = min(_size(rng, 64, 8192), 2 ** 29 // (E * K))
        T = _log_int(rng, 1, max(1, min(4096, 2 ** 38 // (N * K * k))))
        return dict(op=op, dtype=dtype, T=T, k=k, E=E, N=N, K=K, gather=rng.random() < 0.5, bias=rng.random() < 0.3)
    if op == "route":
        return dict(op=op, dtype=rng.choice(["bf16", "fp16", "fp32"]), T=_log_int(rng, 1, min(16384, 2 ** 22 // E)),
                    k=k, E=E, renormalize=rng.random() < 0.5)
    d = _size(rng, 64, 16384)
    if op == "combine":
        return dict(op=op, dtype=dtype, T=_log_int(rng, 1, min(4096, 2 ** 28 // (d * k))), k=k, d=d,
                    addend=rng.random() < 0.5)
    if op == "act":
        return dict(op=op, dtype=dtype, M=_log_int(rng, 1, min(32768, 2 ** 25 // d)), d=d)
    return dict(op=op, dtype=dtype, M=_log_int(rng, 1, min(8192, 2 ** 26 // d)), d=d, y=rng.random() < 0.5)


def _blocks(d):
    return -(-d // BLOCK)


def _codes_like(*shape):
    """A buffer of e4m3 codes whose rows start at 16-byte boundaries."""
    return torch.zeros(*shape[:-1], -(-shape[-1] // 16) * 16, dtype=F8, device=DEVICE)[..., :shape[-1]]


def _scales_like(M, d):
    """A buffer of block scales whose rows start at 16-byte boundaries."""
    return torch.zeros(M, -(-_blocks(d) // 4) * 4, device=DEVICE)[:, :_blocks(d)]


def _router_logits(T, E, g):
    """Logits of a router some of whose experts are chosen more often than others."""
    popular = torch.randn(E, generator=g, device=DEVICE) * 0.5
    return torch.randn(T, E, generator=g, device=DEVICE) * 1.5 + popular


def _sort_by_expert(experts, E):
    """offsets [E + 1], rows and place of the experts chosen [T, k], rows of an expert in the tokens' order."""
    T, k = experts.shape
    flat = experts.reshape(-1)
    order = torch.sort(flat, stable=True).indices
    count = (flat[None, :] == torch.arange(E, device=DEVICE, dtype=flat.dtype)[:, None]).sum(1)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=DEVICE)
    offsets[1:] = torch.cumsum(count, 0)
    place = torch.empty_like(order)
    place[order] = torch.arange(T * k, device=DEVICE)
    return offsets, (order // k).to(torch.int32), place.to(torch.int32).reshape(T, k)


def prepare(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)
    dtype, op = TYPES[case["dtype"]], case["op"]
    randn = lambda *size: torch.randn(*size, generator=g, device=DEVICE)  # noqa: E731
    rand = lambda *size: torch.rand(*size, generator=g, device=DEVICE)  # noqa: E731
    s = dict(case, dtype=dtype)
    if op in ("gemm", "grouped"):
        N, K = case["N"], case["K"]
        E = case["E"] if op == "grouped" else 1
        M = case["T"] * case["k"] if op == "grouped" else case["M"]
        if op == "grouped":
            experts = torch.sort(_router_logits(case["T"], E, g), dim=1, descending=True).indices[:, :case["k"]]
            s["offsets"], rows, _ = _sort_by_expert(experts, E)
            s["rows"] = rows if case["gather"] else None
            s["ends"] = s["offsets"].tolist()           # the plain form's: it takes one expert after another
        tokens = case["T"] if op == "grouped" and case["gather"] else M
        s["a"], s["b"] = _codes_like(tokens, K), _codes_like(E, N, K)
        for t in [s["a"], *s["b"]]:
            t.copy_((randn(t.shape) * 150).clamp_(-448, 448))      # blocks whose largest code is near 448
        s["sa"] = _scales_like(tokens, K)
        s["sa"].copy_((rand(tokens, _blocks(K)) + 0.5) * 0.01)
        s["sb"] = (rand(E, _blocks(N), _blocks(K)) + 0.5) * (0.01 / math.sqrt(K))
        s["bias"] = (randn(E, N) * 0.5).to(dtype) if case["bias"] else None
        if op == "gemm":
            s["b"], s["sb"] = s["b"][0], s["sb"][0]
            s["bias"] = s["bias"][0] if case["bias"] else None
        s["c"] = torch.empty(M, N, dtype=dtype, device=DEVICE)
        return s
    if op == "route":
        T, k, E = case["T"], case["k"], case["E"]
        s["logits"] = _router_logits(T, E, g).to(dtype)
        s["weights"] = torch.empty(T, k, device=DEVICE)
        for name, shape in (("experts", (T, k)), ("offsets", (E + 1,)), ("rows", (T * k,)), ("place", (T, k))):
            s[name] = torch.empty(shape, dtype=torch.int32, device=DEVICE)
        return s
    d = case["d"]
    if op == "combine":
        T, k = case["T"], case["k"]
        s["c"] = randn(T * k, d).to(dtype)
        s["place"] = torch.argsort(rand(T * k)).to(torch.int32).reshape(T, k)
        s["weights"] = torch.softmax(randn(T, k), 1)
        s["addend"] = randn(T, d).to(dtype) if case["addend"] else None
        s["y"] = torch.empty(T, d, dtype=dtype, device=DEVICE)
        return s
    M = case["M"]
    nb = _blocks(d)
    s["q"] = torch.zeros(M, nb * BLOCK, dtype=F8, device=DEVICE)   # whole blocks, so that the values are one product
    s["scales"] = _scales_like(M, d)
    s["values"] = torch.empty(M, nb, BLOCK, dtype=dtype, device=DEVICE)
    if op == "act":
        s["gu"] = (randn(M, 2 * d) * 1.5).to(dtype)
        return s
    # a residual stream: larger than a layer's output, with a few channels larger still
    channel = torch.where(rand(d) < 0.002, 20.0, 1.0)
    s["residual"] = (randn(M, d).mul_(3.0).mul_(channel)).to(dtype)
    s["weight"] = (1 + 0.2 * randn(d)).to(dtype)
    s["x"] = randn(M, d).to(dtype)
    s["h"] = torch.empty(M, d, dtype=dtype, device=DEVICE)
    s["y"] = torch.empty(M, d, dtype=dtype, device=DEVICE) if case["y"] else None
    return s


def _in_blocks(u):
    """[M, d] as [M, blocks, 128], the last block filled up with zeros."""
    M, d = u.shape
    full = torch.zeros(M, _blocks(d) * BLOCK, dtype=u.dtype, device=u.device)
    full[:, :d] = u
    return full.view(M, -1, BLOCK)


def _codes(u, factor):
    """Codes of u [M, d], as the values they stand for where u is times `factor` [M, 1], and their scales."""
    M, d = u.shape
    b = _in_blocks(u)
    a = b.abs().amax(2, keepdim=True)
    use = a >= TINY
    code = torch.where(use, b * (448.0 / torch.where(use, a, 1.0)), 0.0).clamp(-448, 448).to(F8).to(u.dtype)
    scale = torch.where(use, a * factor[:, :, None] / 448.0, 0.0)
    return (code * scale).view(M, -1)[:, :d], scale[:, :, 0]


def _values(q, s):
    """Codes q [..., K] with the block scales s spread over them, in 32 bits."""
    K = q.shape[-1]
    return q.to(torch.float32) * s.repeat_interleave(BLOCK, -1)[..., :K]


def _product(a, sa, b, sb, bias):
    w = _values(b, sb.repeat_interleave(BLOCK, -2)[..., :b.shape[-2], :])
    c = torch.matmul(_values(a, sa), w.t())
    return c if bias is None else c + bias.to(torch.float32)


def _run_own(s):
    from quantized_two_stage_amd import qr
    op = s["op"]
    if op == "gemm":
        qr.qr_gemm_f8(s["a"], s["sa"], s["b"], s["sb"], s["c"], bias=s["bias"])
        return {"c": s["c"]}
    if op == "grouped":
        qr.qr_gemm_f8_grouped(s["a"], s["sa"], s["b"], s["sb"], s["offsets"], s["c"], rows=s["rows"], bias=s["bias"])
        return {"c": s["c"]}
    if op == "route":
        if "workspace" not in s:        # kept with the layer, as its weights are
            s["workspace"] = qr.alloc_route_workspace(s["T"], s["E"], s["k"])
        qr.qr_route(s["logits"], s["weights"], s["experts"], s["offsets"], s["rows"], s["place"],
                    renormalize=s["renormalize"], workspace=s["workspace"])
        return {name: s[name] for name in ("weights", "experts", "offsets", "rows", "place")}
    if op == "combine":
        qr.qr_combine(s["c"], s["place"], s["weights"], s["y"], addend=s["addend"])
        return {"y": s["y"]}
    q = s["q"][:, :s["d"]]
    out = {}
    if op == "act":
        qr.qr_silu_mul_f8(s["gu"], q, s["scales"])
    else:
        qr.qr_add_rmsnorm_f8(s["x"], s["residual"], s["weight"], EPS, s["h"], s["y"], q, s["scales"])
        out = {"h": s["h"]} if s["y"] is None else {"h": s["h"], "y": s["y"]}
    torch.mul(s["q"].to(s["dtype"]).view(s["values"].shape), s["scales"][:, :, None], out=s["values"])
    return dict(out, values=s["values"].view(s["M"], -1)[:, :s["d"]], scales=s["scales"])


def run(s):
    if own:
        return _run_own(s)
    op, real = s["op"], torch.float32
    if op == "gemm":
        return {"c": _product(s["a"], s["sa"], s["b"], s["sb"], s["bias"]).to(s["dtype"])}
    if op == "grouped":
        c = torch.empty_like(s["c"])
        for e, (lo, hi) in enumerate(zip(s["ends"], s["ends"][1:])):
            if lo < hi:
                at = slice(lo, hi) if s["rows"] is None else s["rows"][lo:hi].long()
                c[lo:hi] = _product(s["a"].view(torch.uint8)[at].view(F8), s["sa"][at], s["b"][e], s["sb"][e],
                                    None if s["bias"] is None else s["bias"][e]).to(s["dtype"])
        return {"c": c}
    if op == "route":
        logits = s["logits"].to(real)
        top, experts = torch.sort(logits, dim=1, descending=True, stable=True)
        experts = experts[:, :s["k"]].to(torch.int32)
        among = top[:, :s["k"]] if s["renormalize"] else top
        e = torch.exp(among - top[:, :1])
        weights = e[:, :s["k"]] / e.sum(1, keepdim=True)
        offsets, rows, place = _sort_by_expert(experts, s["E"])
        return {"weights": weights, "experts": experts, "offsets": offsets, "rows": rows, "place": place}
    if op == "combine":
        y = torch.zeros(s["T"], s["d"], dtype=real, device=DEVICE)
        for j in range(s["k"]):
            y += s["weights"][:, j:j + 1] * s["c"][s["place"][:, j].long()].to(real)
        if s["addend"] is not None:
            y += s["addend"].to(real)
        return {"y": y.to(s["dtype"])}
    out = {}
    if op == "act":
        gate, up = s["gu"][:, :s["d"]].to(real), s["gu"][:, s["d"]:].to(real)
        u = gate / (1 + torch.exp(-gate)) * up
        factor = torch.ones_like(u[:, :1])
    else:
        out["h"] = (s["x"].to(real) + s["residual"].to(real)).to(s["dtype"])
        h = out["h"].to(real)
        factor = torch.rsqrt((h * h).sum(1, keepdim=True) / s["d"] + EPS)
        u = h * s["weight"].to(real)
        if s["y"] is not None:
            out["y"] = (u * factor).to(s["dtype"])
    values, scales = _codes(u, factor)
    return dict(out, values=values.to(s["dtype"]), scales=scales)


def _round_e4m3(t):
    """t (64 bits, |t| <= 448) to the nearest e4m3 value, ties to even."""
    exponent = torch.frexp(t).exponent - 1                # of the leading bit
    step = torch.ldexp(torch.ones_like(t), exponent.clamp(min=-6) - 3)
    return torch.round(t / step) * step


def exact(case, seed):
    """The same from the definition in 64 bits; nothing is rounded but what the definition rounds (the sum with the
    residual, the codes)."""
    s = prepare(case, seed)
    f64 = torch.float64
    op = s["op"]
    if op in ("gemm", "grouped"):
        K, N = s["K"], s["N"]
        block = torch.arange(K, device=DEVICE) // BLOCK
        channel = torch.arange(N, device=DEVICE) // BLOCK
        M = s["c"].shape[0]
        ends = s["ends"] if op == "grouped" else [0, M]
        token = torch.arange(M, device=DEVICE)
        if op == "grouped" and s["gather"]:
            token = s["rows"].long()
        a64 = s["a"].to(f64) * s["sa"].to(f64)[:, block]
        c = torch.empty(M, N, dtype=f64, device=DEVICE)
        for e in range(len(ends) - 1):
            lo, hi = ends[e], ends[e + 1]
            if lo == hi:
                continue
            one = (lambda t: t[e]) if op == "grouped" else (lambda t: t)
            w = (one(s["b"]).to(f64) * one(s["sb"]).to(f64)[channel][:, block]).t().contiguous()
            for i in range(lo, hi, 2048):
                c[i:min(i + 2048, hi)] = a64[token[i:min(i + 2048, hi)]] @ w
            if s["bias"] is not None:
                c[lo:hi] += one(s["bias"]).to(f64)
        return {"c": c}
    if op == "route":
        T, k, E = s["T"], s["k"], s["E"]
        logits = s["logits"].to(f64)
        # an expert's rank: how many lie above it, or are equal and before it
        index = torch.arange(E, device=DEVICE)
        experts = torch.empty(T, k, dtype=torch.long, device=DEVICE)
        for i in range(0, T, 64):
            x = logits[i:i + 64]
            above = (x[:, None, :] > x[:, :, None]) | ((x[:, None, :] == x[:, :, None]) & (index < index[:, None]))
            experts[i:i + 64] = torch.argsort(above.sum(2), dim=1)[:, :k]
        chosen = logits.gather(1, experts)
        weights = torch.softmax(chosen, 1) if s["renormalize"] else torch.softmax(logits, 1).gather(1, experts)
        flat = experts.reshape(-1)
        order = torch.argsort(flat * (T * k) + torch.arange(T * k, device=DEVICE))
        offsets = torch.bucketize(torch.arange(E + 1, device=DEVICE), flat[order])
        i32 = torch.int32
        return {"weights": weights, "experts": experts.to(i32), "offsets": offsets.to(i32),
                "rows": (order // k).to(i32), "place": torch.argsort(order).to(i32).view(T, k)}
    if op == "combine":
        y = (s["weights"].to(f64)[:, None, :] @ s["c"][s["place"].long()].to(f64))[:, 0]
        return {"y": y if s["addend"] is None else y + s["addend"].to(f64)}
    out = {}
    d = s["d"]
    if op == "act":
        gate, up = s["gu"].to(f64).split(d, dim=1)
        u = gate * torch.sigmoid(gate) * up
        gain = 1.0
    else:
        out["h"] = (s["x"].to(f64) + s["residual"].to(f64)).to(s["dtype"]).to(f64)
        gain = out["h"].square().mean(1, keepdim=True).add(EPS).pow(-0.5)
        u = out["h"] * s["weight"].to(f64)
        if s["y"] is not None:
            out["y"] = u * gain
    values, scales = torch.empty_like(u), torch.empty(s["M"], _blocks(d), dtype=f64, device=DEVICE)
    for b in range(_blocks(d)):
        part = u[:, b * BLOCK:(b + 1) * BLOCK]
        largest = part.abs().amax(1, keepdim=True)
        code = torch.where(largest > 0, _round_e4m3(448 * part / largest), 0.0)
        scales[:, b:b + 1] = largest * gain / 448
        values[:, b * BLOCK:(b + 1) * BLOCK] = code * scales[:, b:b + 1]
    return dict(out, values=values, scales=scales)


def work(case):
    op = case["op"]
    if op in ("gemm", "grouped"):
        N, K = case["N"], case["K"]
        M, rows, hit = (case["M"], case["M"], 1) if op == "gemm" else (
            case["T"] * case["k"], case["T"] * (1 if case["gather"] else case["k"]),
            # experts hit, were all chosen alike
            case["E"] * (1 - (1 - case["k"] / case["E"]) ** case["T"]))
        return {"bytes": int(rows * (K + 4 * _blocks(K)) + hit * (N * K + 4 * _blocks(N) * _blocks(K)
                                                                  + (2 * N if case["bias"] else 0)) + 2 * M * N),
                "flops": 2 * M * N * K}
    if op == "route":
        T, k, E = case["T"], case["k"], case["E"]
        return {"bytes": T * E * (4 if case["dtype"] == "fp32" else 2) + 16 * T * k + 4 * (E + 1), "flops": 4 * T * E}
    d = case["d"]
    if op == "combine":
        T, k = case["T"], case["k"]
        return {"bytes": 2 * T * d * (k + 1 + case["addend"]) + 8 * T * k, "flops": 2 * T * k * d}
    M = case["M"]
    codes = M * d + 4 * M * _blocks(d)
    if op == "act":
        return {"bytes": 4 * M * d + codes, "flops": 12 * M * d}
    return {"bytes": 2 * M * d * (3 + case["y"]) + 2 * d + codes, "flops": 10 * M * d}
