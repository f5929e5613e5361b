"""The operators of include/qr_f8.h on the GPU at the ends of what their header promises (tolerances: test_f8_gpu.py)."""
import pytest
import torch

import f8_tiles
from f8_edges import GRAPH_DENSE, GRAPH_GROUPED, LONG, MANY, ROUTES
from test_f8_gpu import (F8, INF, NAN, TYPES, blocks, check_product, check_route, codes, qr, reference, route,  # noqa: F401
                         rows_in, say, scales_like, sizes_of_groups)

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


@pytest.mark.parametrize("M,N,K", GRAPH_DENSE)
def test_captured_product(qr, M, N, K):  # noqa: F811
    """a product in a graph takes what its inputs hold at each replay; on another stream than theirs too"""
    say("captured", M, N, K)
    g = torch.Generator(device="cuda").manual_seed(M + N + K)

    def inputs():
        return [codes(M, K, g), scales_like(M, K, g), codes(N, K, g), scales_like(blocks(N), K, g),
                torch.randn(N, generator=g, device="cuda").half()]

    held = inputs()
    c, eager = torch.empty(M, N, dtype=torch.float16, device="cuda"), torch.empty(M, N, dtype=torch.float16, device="cuda")
    qr.qr_gemm_f8(*held[:4], eager, bias=held[4])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qr.qr_gemm_f8(*held[:4], c, bias=held[4])
    for i in range(4):
        new = inputs()
        for t, n in zip(held, new):
            t.copy_(n)
        c.fill_(9.0)
        graph.replay()
        torch.cuda.synchronize()
        check_product(c, *reference(*new), (M, N, K, i))
        qr.qr_gemm_f8(*held[:4], eager, bias=held[4])         # eager work between the replays
        assert torch.equal(c, eager)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    c.fill_(9.0)
    torch.cuda.synchronize()
    qr.qr_gemm_f8(*held[:4], c, bias=held[4], stream=side)
    side.synchronize()
    assert torch.equal(c, eager)


@pytest.mark.parametrize("T,k,E,N,K", GRAPH_GROUPED)
def test_captured_groups_follow_the_router(qr, T, k, E, N, K):  # noqa: F811
    """the router, its experts' product over the tokens in place and the weighted sum in one graph: other logits give other
    offsets and rows, the same graph the new product"""
    say("captured groups", T, k, E, N, K)
    g = torch.Generator(device="cuda").manual_seed(T + E + N + K)
    i32 = dict(dtype=torch.int32, device="cuda")
    M = T * k
    logits = torch.zeros(T, E, device="cuda")
    weights, experts, offsets = torch.empty(T, k, device="cuda"), torch.empty(T, k, **i32), torch.empty(E + 1, **i32)
    rows, place, ws = torch.empty(M, **i32), torch.empty(T, k, **i32), qr.alloc_route_workspace(T, E, k)
    a, sa = codes(T, K, g), scales_like(T, K, g)
    b, sb = codes(E * N, K, g).unflatten(0, (E, N)), scales_like(E * blocks(N), K, g).unflatten(0, (E, blocks(N)))
    c, y = torch.empty(M, N, dtype=torch.bfloat16, device="cuda"), torch.empty(T, N, dtype=torch.bfloat16, device="cuda")

    def run(stream=None):
        qr.qr_route(logits, weights, experts, offsets, rows, place, renormalize=True, workspace=ws, stream=stream)
        qr.qr_gemm_f8_grouped(a, sa, b, sb, offsets, c, rows=rows, stream=stream)
        qr.qr_combine(c, place, weights, y, stream=stream)

    def result():
        torch.cuda.synchronize()
        return [t.clone() for t in (weights, experts, offsets, rows, place, c, y)]

    run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    before = None
    for i in range(4):
        popular = torch.randn(E, generator=g, device="cuda") * i            # more and more unequal
        logits.copy_(torch.randn(T, E, generator=g, device="cuda") + popular)
        a.view(torch.uint8).copy_(codes(T, K, g).view(torch.uint8))
        for t, fill in ((weights, NAN), (experts, 0), (offsets, 0), (rows, 0), (place, 0), (c, NAN), (y, NAN)):
            t.fill_(fill)
        graph.replay()
        got = result()
        run()                                                              # eager work between the replays
        for x, want in zip(got, result()):
            assert torch.equal(x, want)
        assert int(offsets[0]) == 0 and int(offsets[-1]) == M
        assert torch.equal(torch.bincount(experts.reshape(-1).long(), minlength=E), (offsets[1:] - offsets[:-1]).long())
        assert before is None or not torch.equal(before, offsets)
        before = offsets.clone()
        check_groups(c, a, sa, rows, b, sb, offsets, (T, k, E, N, K, i))
        exact = (weights.double()[:, :, None] * c.double()[place.long()]).sum(1)
        size = (weights.double()[:, :, None] * c.double()[place.long()].abs()).sum(1)
        tol = (k + 1) * 2.0 ** -24 * size
        assert bool(((y.double() - exact).abs() <= tol + 2.0 ** -8 * (exact.abs() + tol) + 2.0 ** -134).all())
    want = result()
    c.fill_(NAN)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    run(side)
    side.synchronize()
    for x, w in zip(result(), want):
        assert torch.equal(x, w)


@pytest.mark.parametrize("dtype", ["fp16", "bf16", "fp32"])
@pytest.mark.parametrize("T,E,k", ROUTES)
def test_route_in_every_kernel(qr, T, E, k, dtype):  # noqa: F811
    """values that lie close together, so that 16-bit ones are often equal, and some that are not numbers"""
    g = torch.Generator(device="cuda").manual_seed(T + E + k)
    for renormalize in (False, True):
        say("route", T, E, k, dtype, renormalize)
        logits = torch.randn(T, E + 5, generator=g, device="cuda").to(TYPES[dtype])[:, 2:E + 2]
        if T > 4:
            logits[0] = -INF
            logits[1, E - 1], logits[2, 0] = NAN, INF
            logits[3, ::2] = -INF
            logits[4] = 0.0
        check_route(logits, k, renormalize, route(qr, logits, k, renormalize), (T, E, k, dtype, renormalize))
