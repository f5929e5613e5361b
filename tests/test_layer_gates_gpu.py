"""qr_silu_mul_q8 over every finite 16-bit gate, in each of its row kernels, against 64 bits: gates beside ordinary ones,
and rows whose gates are all the same (where the row's scale is as small as the gate makes it).

Tolerance, derived before the first run (e = 2^-24, half a unit in the last place of binary32): exp(-|g|) is v_exp_f32's
(one unit, 2e) times a correction (e); the product with g, 1 + exp, the corrected quotient and the product with u are
within e each: 7e.  Beyond 64 (where 1 + exp is 1 and the quotient exact: 5e) u is first multiplied by |g|/64 (e) and, for
negative gates, twice by the root of exp(g + 64): 2 * (3e + e) more.  So v is within 14e of its value, whatever the gate,
counted as 16e, or within 2^-148 where it is subnormal; the largest magnitude a likewise, the scale a/127 within e more,
and the code, of the exact quotient of these, within half a step and 127 * 2 * 16e (and the comparison's own roundings)."""
import pytest
import torch

from test_layer_gpu import qr  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu

E = 2.0 ** -24
OFF = 16 * E
TINY, TOP = 2.0 ** -119, 3.4028234663852886e38
TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


def finite_values(t):
    v = torch.arange(65536, dtype=torch.int32, device="cuda").to(torch.int16).view(t)
    return v[v.isfinite()]


def run_and_check(qr, g, u, label):  # noqa: F811
    print(label, tuple(g.shape), flush=True)
    M, d = g.shape
    q, s = qr.alloc_q8(M, d)
    qr.qr_silu_mul_q8(torch.cat([g, u], 1), q, s)
    torch.cuda.synchronize()
    for i in range(0, M, 4096):
        check(g[i:i + 4096].double(), u[i:i + 4096].double(), q[i:i + 4096].double(), s[i:i + 4096].double(),
              g[i:i + 4096, 0], label)


def check(g, u, q, s, first, label):
    e = torch.exp(-g.abs())
    v = torch.where(g < 0, g * e, g) / (1 + e) * u
    a = v.abs().amax(1)

    def none(bad, what):
        assert not bool(bad.any()), (label, what, int(bad.sum()), first[bad][:8].tolist(), s[bad][:8].tolist())

    over, zero = a > TOP, a < TINY
    edge = ((a / TOP - 1).abs() < 2 * OFF) | ((a / TINY - 1).abs() < 2 * OFF)
    none(over & ~edge & ~(s.isnan() & (q == 0).all(1)), "past the largest value, but not NaN")
    none(zero & ~edge & ~((s == 0) & (q == 0).all(1)), "below 2^-119, but not zero")
    fine = ~over & ~zero & ~edge
    none(fine & ~s.isfinite(), "scale of a finite row")
    none(fine & ((s * 127 - a).abs() > (OFF + 2 * E) * a), "scale")
    size = torch.where(fine, a, torch.ones_like(a))[:, None]
    none(fine & (q.abs().amax(1) != 127), "largest code")
    off = (q - 127 * v / size).abs().amax(1)
    none(fine & (off > 0.5 + 127 * (2 * OFF + 2.0 ** -148 / size[:, 0]) + 1e-9), "codes")


def signs(size, gen):
    return torch.randint(0, 2, size, generator=gen, device="cuda") * 2.0 - 1


# a wave to a row, whole and short; a workgroup; the two passes of rows below 8
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("d", [5, 64, 67, 520, 523])
def test_each_gate_beside_ordinary_ones(qr, d, dtype):  # noqa: F811
    t = TYPES[dtype]
    gates = finite_values(t)
    gen = torch.Generator(device="cuda").manual_seed(d)
    M = gates.numel()
    g = (2 * torch.randn(M, d, generator=gen, device="cuda")).to(t)
    at = torch.randint(0, d, (M,), generator=gen, device="cuda")
    g[torch.arange(M, device="cuda"), at] = gates
    # below 1, so that the largest gates stay below the largest binary32
    u = ((0.25 + 0.75 * torch.rand(M, d, generator=gen, device="cuda")) * signs((M, d), gen)).to(t)
    run_and_check(qr, g, u, ("beside", d, dtype))


# two and four vectors a lane, whole and short, and two passes
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("d", [8200, 8203, 16392, 16395, 32776, 40003])
def test_gates_in_long_rows(qr, d, dtype):  # noqa: F811
    """every gate, 1024 to a row in the order of their magnitude, scattered among ordinary ones"""
    t = TYPES[dtype]
    gates = finite_values(t)
    gates = gates[gates.float().abs().argsort(stable=True)]
    M, gen = -(-gates.numel() // 1024), torch.Generator(device="cuda").manual_seed(d)
    g = (2 * torch.randn(M, d, generator=gen, device="cuda")).to(t)
    for m in range(M):
        some = gates[1024 * m:1024 * (m + 1)]
        g[m, torch.randperm(d, generator=gen, device="cuda")[:some.numel()]] = some
    u = ((0.25 + 0.75 * torch.rand(M, d, generator=gen, device="cuda")) * signs((M, d), gen)).to(t)
    run_and_check(qr, g, u, ("long", d, dtype))


@pytest.mark.parametrize("d", [7, 72, 515])
@pytest.mark.parametrize("dtype,low,high", [("fp16", -1, 1), ("fp16", -12, 15.9), ("bf16", -1, 1), ("bf16", -12, 15.9),
                                            ("bf16", -60, 60), ("bf16", 100, 127.9)])
def test_rows_of_one_gate(qr, d, dtype, low, high):  # noqa: F811
    """the gate alone decides how large a row is: up to 2^16 times the smallest, and, in bfloat16, beyond"""
    t = TYPES[dtype]
    gates = finite_values(t)
    gen = torch.Generator(device="cuda").manual_seed(d)
    M = gates.numel()
    size = torch.exp2(low + (high - low) * torch.rand(M, d, generator=gen, device="cuda", dtype=torch.float64))
    u = (size * signs((M, d), gen)).clamp(-torch.finfo(t).max, torch.finfo(t).max).to(t)
    run_and_check(qr, gates[:, None].expand(M, d), u, ("one gate", d, dtype, low, high))


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("d", [2056, 9000, 20001, 33000])
def test_long_rows_of_one_gate(qr, d, dtype):  # noqa: F811
    t = TYPES[dtype]
    gates = finite_values(t)
    size = gates.float().abs()
    far = gates[(size > 78) & (size < 110)]
    gates = torch.cat([far[::max(1, far.numel() // 100)], gates[::997]])
    M, gen = gates.numel(), torch.Generator(device="cuda").manual_seed(d)
    u = (torch.exp2(28 * torch.rand(M, d, generator=gen, device="cuda") - 12.5) * signs((M, d), gen)).to(t)
    run_and_check(qr, gates[:, None].expand(M, d), u, ("one gate", d, dtype))


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("d", [6, 64, 2000, 9000, 20000, 33000])
def test_infinities_and_nan_stay(qr, d, dtype):  # noqa: F811
    """a row with an infinity or a NaN has codes 0 and scale NaN, whatever the other half holds there"""
    t = TYPES[dtype]
    inf, nan = float("inf"), float("nan")
    pairs = [(inf, 1.0), (-inf, 1.0), (inf, 0.0), (-inf, 0.0), (nan, 1.0), (nan, 0.0), (1.0, inf), (0.0, inf),
             (-85.0, inf), (-85.0, -inf), (-95.0, inf), (-1000.0, inf), (-95.0, nan), (-1000.0, nan), (1000.0, nan),
             (-inf, inf), (nan, nan), (-inf, nan), (inf, -inf)]
    gu = torch.randn(len(pairs) + 1, 2 * d, generator=torch.Generator("cuda").manual_seed(d), device="cuda").to(t)
    for m, (g, u) in enumerate(pairs):
        gu[m, (3 * m) % d], gu[m, d + (3 * m) % d] = g, u
    q, s = qr.alloc_q8(gu.shape[0], d)
    q.fill_(1)
    qr.qr_silu_mul_q8(gu, q, s)
    torch.cuda.synchronize()
    n = len(pairs)
    assert bool(s[:n].isnan().all()) and not bool(q[:n].any())
    assert bool(s[n].isfinite()) and int(q[n].abs().max()) == 127
