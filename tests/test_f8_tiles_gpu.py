"""The products in 8-bit floating point in every tile, with sums that end everywhere in its ring and in the parts in
which scales come, against 64 bits (tolerances: test_f8_gpu.py).  Which sizes take which tile is asked of the launch's
own rule."""
import pytest
import torch

import f8_tiles
from test_f8_gpu import blocks, check_product, codes, qr, reference, rows_in, say, scales_like, sizes_of_groups  # noqa: F401
from test_f8_tile_choice import EDGES

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tile", range(10))
def test_one_product(qr, tile):  # noqa: F811
    for K in EDGES:
        if tile not in f8_tiles.smallest(K, 0):
            continue
        M, N = f8_tiles.smallest(K, 0)[tile]
        say("tile", tile, M, N, K)
        g = torch.Generator(device="cuda").manual_seed(M + N + K)
        a, sa = codes(M, K, g), scales_like(M, K, g)
        b, sb = codes(N, K, g), scales_like(blocks(N), K, g)
        bias = torch.randn(N, generator=g, device="cuda").half()
        _, c = rows_in(M, N, N + 1, torch.float16, 9.0)
        qr.qr_gemm_f8(a, sa, b, sb, c, bias=bias)
        check_product(c, *reference(a, sa, b, sb, bias), (tile, M, N, K))


@pytest.mark.parametrize("E", [1, 8, 70])
@pytest.mark.parametrize("tile", range(10))
def test_groups(qr, tile, E):  # noqa: F811
    for K in EDGES:
        if tile not in f8_tiles.smallest(K, E):
            continue
        M, N = f8_tiles.smallest(K, E)[tile]
        say("tile", tile, E, M, N, K)
        g = torch.Generator(device="cuda").manual_seed(E + M + N + K)
        tokens = max(1, M // 2)
        a, sa = codes(tokens, K, g), scales_like(tokens, K, g)
        b, sb = codes(E * N, K, g).unflatten(0, (E, N)), scales_like(E * blocks(N), K, g).unflatten(0, (E, blocks(N)))
        offsets = sizes_of_groups("random", E, M, g)
        rows = torch.randint(0, tokens, (M,), generator=g, device="cuda").to(torch.int32)
        _, c = rows_in(M, N, N + 1, torch.bfloat16, 9.0)
        qr.qr_gemm_f8_grouped(a, sa, b, sb, offsets, c, rows=rows)
        ends = offsets.tolist()
        for e in range(E):
            lo, hi = ends[e], ends[e + 1]
            if lo < hi:
                at = rows[lo:hi].long()
                check_product(c[lo:hi], *reference(a.view(torch.uint8)[at].view(a.dtype), sa[at], b[e], sb[e], None),
                              (tile, E, M, N, K, e))
