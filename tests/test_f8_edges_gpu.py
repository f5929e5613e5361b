"""The operators of include/qr_f8.h on the GPU at the ends of what their header promises (tolerances: test_f8_gpu.py)."""
import pytest
import torch

import f8_tiles
from f8_edges import LONG, MANY
from test_f8_gpu import (F8, blocks, check_product, codes, qr, reference, rows_in, say, scales_like,  # noqa: F401
                         sizes_of_groups)

pytestmark = pytest.mark.gpu


def check_groups(c, a, sa, rows, b, sb, offsets, label):
    ends = offsets.tolist()
    for e in range(b.shape[0]):
        lo, hi = ends[e], ends[e + 1]
        if lo < hi:
            at = rows[lo:hi].long()
            check_product(c[lo:hi], *reference(a.view(torch.uint8)[at].view(F8), sa[at], b[e], sb[e], None), (*label, e))


@pytest.mark.parametrize("kind", ["random", "short"])
@pytest.mark.parametrize("E,M,N,K", MANY)
def test_large_tiles_of_many_experts(qr, E, M, N, K, kind):  # noqa: F811
    """more experts than a wave adds up at a time, in tiles of 256 x 256"""
    say("many experts", E, M, N, K, kind)
    g = torch.Generator(device="cuda").manual_seed(E + M + N + K)
    tokens = M // 3
    a, sa = codes(tokens, K, g), scales_like(tokens, K, g)
    b, sb = codes(E * N, K, g).unflatten(0, (E, N)), scales_like(E * blocks(N), K, g).unflatten(0, (E, blocks(N)))
    offsets = sizes_of_groups(kind, E, M, g)
    rows = torch.randint(0, tokens, (M,), generator=g, device="cuda").to(torch.int32)
    _, c = rows_in(M, N, N + 1, torch.bfloat16, 9.0)
    qr.qr_gemm_f8_grouped(a, sa, b, sb, offsets, c, rows=rows)
    lo, hi = int(offsets[0]), int(offsets[-1])
    assert bool((c[:lo] == 9.0).all()) and bool((c[hi:] == 9.0).all())
    check_groups(c, a, sa, rows, b, sb, offsets, (E, M, N, K))


def uneven(rows, K, g):
    """block scales over six powers of two, so that another block's would be far off"""
    s = scales_like(rows, K, g)
    return s.copy_(0.005 * torch.exp2(6 * torch.rand(s.shape, generator=g, device="cuda") - 3))


@pytest.mark.parametrize("tile,K", LONG)
def test_long_sums(qr, tile, K):  # noqa: F811
    """more than 128 blocks: every buffer of the scales is filled again and read again"""
    M, N = f8_tiles.smallest(K, 0)[tile]
    say("long", tile, M, N, K)
    g = torch.Generator(device="cuda").manual_seed(M + N + K)
    a, sa = codes(M, K, g), uneven(M, K, g)
    b, sb = codes(N, K, g), uneven(blocks(N), K, g)
    _, c = rows_in(M, N, N + 1, torch.float16, 9.0)
    qr.qr_gemm_f8(a, sa, b, sb, c)
    check_product(c, *reference(a, sa, b, sb, None), (tile, M, N, K))
    # the test can fail: with the scales that a buffer held before (16 blocks back the tokens', 128 the weights') most
    # outputs would be out of tolerance (the weights' where more than the 16 codes of K = 16400 are that far on)
    stale = [(sa.roll(16, 1), sb), (sa, torch.cat([sb[:, :128], sb[:, :-128]], 1))]
    for x, y in stale[:2 if blocks(K) >= 192 else 1]:
        want, tol = reference(a, x, b, y, None)
        assert bool(((c.double() - want).abs() > tol + 2.0 ** -11 * (want.abs() + tol) + 2.0 ** -25).float().mean() > 0.5)
    if K > 40000:
        return
    E = 8
    M, N = f8_tiles.smallest(K, E)[tile]
    say("long, grouped", tile, M, N, K)
    tokens = max(1, M // 2)
    a, sa = codes(tokens, K, g), uneven(tokens, K, g)
    b, sb = codes(E * N, K, g).unflatten(0, (E, N)), uneven(E * blocks(N), K, g).unflatten(0, (E, blocks(N)))
    offsets = sizes_of_groups("random", E, M, g)
    rows = torch.randint(0, tokens, (M,), generator=g, device="cuda").to(torch.int32)
    _, c = rows_in(M, N, N + 1, torch.float16, 9.0)
    qr.qr_gemm_f8_grouped(a, sa, b, sb, offsets, c, rows=rows)
    check_groups(c, a, sa, rows, b, sb, offsets, (tile, M, N, K))


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
