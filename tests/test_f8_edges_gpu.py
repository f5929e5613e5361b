"""The operators of include/qr_f8.h on the GPU at the ends of what their header promises (tolerances: test_f8_gpu.py)."""
import pytest
import torch

from test_f8_gpu import F8, qr, say  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M", [1, 20, 300])
@pytest.mark.parametrize("large,other,scale,bound", [
    # 2^16 + 7 * 7.5, cut at 8: 2^16 is left, times 2^-6
    ((256.0, 256.0), (1.0, 7.5), 2.0 ** -6, 7 * 2.0 ** -13),
    # 2^-1 + 7 * 1.875 * 2^-12, cut at 2^-11 (2^-13 of 2^-6 * 2^8): 2^-1 is left, times 2^11
    ((2.0 ** -9, 256.0), (2.0 ** -9, 0.234375), 2.0 ** 11, 8 * 7 * 2.0 ** -13),
])
def test_what_an_outlier_costs_its_group(qr, M, large, other, scale, bound):  # noqa: F811
    """one product and seven below the cut: these are lost, which is near the header's bound and far above what sums of
    like products lose"""
    say("outlier", M, large)
    a, b = torch.full((M, 16), 0.0, device="cuda"), torch.full((33, 16), 0.0, device="cuda")
    a[:, :8], b[:, :8] = other[0], other[1]
    a[:, 3], b[:, 3] = large
    sa, sb = torch.full((M, 4), scale, device="cuda")[:, :1], torch.ones(1, 1, device="cuda")
    c = torch.zeros(M, 33, dtype=torch.float16, device="cuda")
    qr.qr_gemm_f8(a.to(F8), sa, b.to(F8), sb, c)
    kept, all_of_it = large[0] * large[1], large[0] * large[1] + 7 * other[0] * other[1]
    assert bool((c == kept * scale).all()) and kept * scale == 1024
    lost = 1 - kept / all_of_it
    assert 0.85 * bound < lost < bound
