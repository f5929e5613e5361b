"""Codes at ties, where round-half-even(127 * u / a) rests on the exact quotient: rows whose largest value is 254 times a
number w that has no short reciprocal, so that every odd multiple of w is a tie while 127 / a is rounded.  The codes are
whole numbers and equal to the formula's in exact fractions."""
from fractions import Fraction

import pytest
import torch

from test_layer_gpu import qr  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu

TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


def half_even(x):
    return int(round(x))                   # Python rounds a Fraction half to even


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("d", [509, 512, 5000, 9000, 20000, 40000])
def test_ties(qr, d, dtype):  # noqa: F811
    t = TYPES[dtype]
    h = torch.arange(d, device="cuda") % 509 - 254            # -254 .. 254, each in every row
    x = h.to(t)[None].expand(6, d).contiguous()
    x[1:, 3::11] = 0
    for w in (1.0, 3.0, 0.8203125, 1.6796875, 0.01116943359375):
        w = float(torch.tensor(w).to(t))
        weight = torch.full((d,), w, dtype=t, device="cuda")
        q, s = qr.alloc_q8(6, d)
        qr.qr_add_rmsnorm_q8(x, None, weight, 1e-5, None, q, s)
        torch.cuda.synchronize()
        code = {i: half_even(Fraction(127 * i, 254)) for i in range(-254, 255)}
        want = torch.tensor([code[int(v)] for v in x[0].tolist()], dtype=torch.int8, device="cuda")
        want = torch.where(x == 0, 0, want[None]).to(torch.int8)
        assert torch.equal(q, want), (d, dtype, w)


def test_products_near_ties(qr):  # noqa: F811
    """values and weights of 11 bits each: a million codes against exact fractions' (64 bits decide all but ties, which
    have a whole numerator)"""
    g = torch.Generator(device="cuda").manual_seed(8)
    M, d = 256, 4096
    x = torch.randint(-2047, 2048, (M, d), generator=g, device="cuda").to(torch.float16)
    w = torch.randint(1024, 2048, (d,), generator=g, device="cuda").to(torch.float16)
    q, s = qr.alloc_q8(M, d)
    qr.qr_add_rmsnorm_q8(x, None, w, 1e-5, None, q, s)
    torch.cuda.synchronize()
    u = x.to(torch.int64) * w.to(torch.int64)
    a = u.abs().amax(1, keepdim=True)
    # round-half-even(127u/a) = (254u + a) // 2a, less one where that is odd and the division leaves nothing
    n = 254 * u + a
    want = torch.div(n, 2 * a, rounding_mode="floor")
    want -= ((n % (2 * a) == 0) & (want % 2 != 0)).to(torch.int64)
    assert torch.equal(q.to(torch.int64), want)
