"""Scales of the norm whose factors are far from 1: a * r / 127 of a finite row is finite wherever the scale itself is, also
where a * r passes the largest binary32 (a large weight on a row with one large value).  Tolerance as in
test_layer_gpu.check_codes."""
import numpy as np
import pytest
import torch

from test_layer_gpu import E, chain, check_codes, norm_reference, qr  # noqa: F401  (qr: a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [7, 64, 504, 2000, 8192, 12000, 16000])
@pytest.mark.parametrize("weight", [3e38, 2e30, 1.0, 1e-30])
def test_one_value_in_a_row(qr, d, weight):  # noqa: F811
    """r = sqrt(d) / |x|, so the scale is weight * sqrt(d) / 127: below the largest binary32 for all of these"""
    x = torch.zeros(5, d, dtype=torch.bfloat16, device="cuda")
    for m, v in enumerate((0.5, -0.99, 1e-3, 1.0, 17.0)):
        x[m, (m * 5) % d] = v
    w = torch.full((d,), weight, dtype=torch.bfloat16, device="cuda")
    if weight == 3e38:
        x[4] *= 0.01                                   # 17 * 3e38 itself would be infinite
    q, s = qr.alloc_q8(5, d)
    qr.qr_add_rmsnorm_q8(x, None, w, 1e-12, None, q, s)
    torch.cuda.synchronize()
    u, r = norm_reference(x, w, float(np.float32(1e-12)))
    assert bool(s.isfinite().all()), (d, weight, s.tolist())
    check_codes(q, s, u, r, (chain(d) / 2 + 6) * E, (d, weight))
