"""The operators of include/qr_f8.h on the GPU at their largest: buffers of more than 4 GiB, more rows than a launch has
workgroups or lanes for (tolerances: test_f8_gpu.py).  What is compared are rows at both ends and where a launch or a pass
over the rows ends; the rest is compared with copies of these rows."""
import pytest
import torch

from test_f8_gpu import (E24, F8, blocks, chain, check_blocks, check_product, codes, qr, reference, say,  # noqa: F401
                         scales_like)

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _memory():
    yield
    torch.cuda.empty_cache()


def repeated(rows, period, fill):
    """[rows, ...] whose row i is row i % period of `fill` [period, ...]"""
    out = torch.empty(rows, *fill.shape[1:], dtype=fill.dtype, device="cuda")
    for i in range(0, rows, period * 64):
        n = min(rows, i + period * 64) - i
        out[i:i + n] = fill.repeat(-(-n // period), *[1] * (fill.dim() - 1))[:n]
    return out


def same_as_first(t, period):
    """every row is that of `period` rows before"""
    step = max(period, (1 << 28) // max(1, t[0].numel()) // period * period)
    again = t[:period].repeat(step // period, *[1] * (t.dim() - 1))
    return all(torch.equal(part, again[:part.shape[0]]) for part in t.split(step))


@pytest.mark.parametrize("d", [7, 520, 1000])
def test_norm_of_more_rows_than_workgroups(qr, d):  # noqa: F811
    M, period = (1 << 21) + 1037, 61
    say("norm", M, d)
    g = torch.Generator(device="cuda").manual_seed(d)
    few = torch.randn(period, d, generator=g, device="cuda").half()
    x = repeated(M, period, few)
    w = (1 + 0.3 * torch.randn(d, generator=g, device="cuda")).half()
    q = torch.zeros(M, d, dtype=torch.uint8, device="cuda")
    s, y = torch.full((M, blocks(d)), 7.0, device="cuda"), torch.zeros(M, d, dtype=torch.float16, device="cuda")
    qr.qr_add_rmsnorm_f8(x, None, w, 1e-5, None, y, q.view(F8), s)
    u = few.double() * w.double()
    r = (few.double().square().mean(1, keepdim=True) + float(torch.tensor(1e-5))).rsqrt()
    check_blocks(q[:period].view(F8), s[:period], u, r, (chain(d) / 2 + 6) * E24, (M, d))
    tol = (chain(d) / 2 + 6) * E24
    exact = u * r
    limit = (2.0 ** -11 + tol) * exact.abs() * (1 + 2.0 ** -11) + 2.0 ** -25
    assert bool(((y[:period].double() - exact).abs() <= limit).all())
    assert same_as_first(q, period) and same_as_first(s, period) and same_as_first(y, period)


def test_activation_of_more_rows_than_a_launch(qr):  # noqa: F811
    d = 16384
    M, period = (1 << 20) + 77, 31                    # 2^31 lanes are 2^20 rows
    say("activation", M, d)
    g = torch.Generator(device="cuda").manual_seed(5)
    gu = repeated(M, period, torch.randn(period, 2 * d, generator=g, device="cuda").bfloat16())
    q, s = torch.zeros(M, d, dtype=torch.uint8, device="cuda"), torch.full((M, d // 128), 7.0, device="cuda")
    qr.qr_silu_mul_f8(gu, q.view(F8), s)
    few, sf = torch.zeros(period, d, dtype=torch.uint8, device="cuda"), torch.zeros(period, d // 128, device="cuda")
    qr.qr_silu_mul_f8(gu[:period], few.view(F8), sf)
    assert torch.equal(few, q[:period]) and torch.equal(sf, s[:period])
    assert same_as_first(q, period) and same_as_first(s, period)
    gate, up = gu[:period].double().split(d, 1)
    v = gate / (1 + torch.exp(-gate)) * up
    a = v.abs().view(period, -1, 128).amax(2)
    assert bool(((sf.double() - a / 448).abs() <= 20 * E24 * a / 448).all())


def test_combination_of_more_tokens_than_a_launch(qr):  # noqa: F811
    d, R, k = 8192, 900000, 2                         # c has 14.7 GB, y 34.4 GB
    T, period = (1 << 21) + 5, 45000
    say("combine", T, d)
    g = torch.Generator(device="cuda").manual_seed(6)
    c = repeated(R, 100, torch.randn(100, d, generator=g, device="cuda").bfloat16())
    place = repeated(T, period, torch.randint(0, R, (period, k), generator=g, device="cuda").to(torch.int32))
    weights = repeated(T, period, torch.randn(period, k, generator=g, device="cuda"))
    y = torch.zeros(T, d, dtype=torch.bfloat16, device="cuda")
    qr.qr_combine(c, place, weights, y)
    for lo, hi in ((0, 2000), ((1 << 21) - 500, T)):
        terms = weights[lo:hi, :, None].double() * c[place[lo:hi].long()].double()
        want, tol = terms.sum(1), (k + 1) * E24 * terms.abs().sum(1)
        assert bool(((y[lo:hi].double() - want).abs() <= tol + 2.0 ** -8 * (want.abs() + tol) + 2.0 ** -134).all())
    assert same_as_first(y, period)


@pytest.mark.parametrize("T,E,k", [(1 << 22, 8, 1), (1 << 19, 64, 8), (1 << 17, 1024, 32)])
@pytest.mark.parametrize("crowd", [False, True])
def test_route_of_many_tokens(qr, T, E, k, crowd):  # noqa: F811
    """the most rows that there may be; with all tokens' first choice the same too"""
    say("route", T, E, k, crowd)
    g = torch.Generator(device="cuda").manual_seed(T + E)
    logits = torch.randn(T, E, generator=g, device="cuda").half()
    if crowd:
        logits[:, E // 2] = 100.0
    i32 = dict(dtype=torch.int32, device="cuda")
    weights = torch.full((T, k), 7.0, device="cuda")
    experts, place = torch.full((T, k), -7, **i32), torch.full((T, k), -7, **i32)
    offsets, rows = torch.full((E + 1,), -7, **i32), torch.full((T * k,), -7, **i32)
    qr.qr_route(logits, weights, experts, offsets, rows, place, workspace=qr.alloc_route_workspace(T, E, k))
    want = torch.empty(T, k, **i32)
    for i in range(0, T, 1 << 16):
        x = logits[i:i + (1 << 16)].float()
        want[i:i + (1 << 16)] = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :k]
    assert torch.equal(experts, want)
    flat = experts.reshape(-1).long()
    order = torch.sort(flat, stable=True).indices
    assert torch.equal(offsets.long()[1:], torch.cumsum(torch.bincount(flat, minlength=E), 0)) and int(offsets[0]) == 0
    assert torch.equal(rows.long(), order // k)
    back = torch.empty_like(order)
    back[order] = torch.arange(T * k, device="cuda")
    assert torch.equal(place.reshape(-1).long(), back)
    for i in (0, T - 5000):
        x = logits[i:i + 5000].double()
        w = torch.softmax(x, 1).gather(1, experts[i:i + 5000].long())
        assert bool(((weights[i:i + 5000].double() - w).abs() <= 34 * E24 * w + 2.0 ** -126).all())


@pytest.mark.parametrize("M,N,K", [(530000, 16, 8192), (530000, 160, 8192), (1 << 20, 2100, 128), (64, 530000, 8208),
                                   (1500, 530000, 8208)])
def test_products_beyond_4_gib(qr, M, N, K):  # noqa: F811
    """of a, of c, of b"""
    say("gemm", M, N, K)
    g = torch.Generator(device="cuda").manual_seed(M + N + K)
    period = 128 * 7                                 # whole blocks of scales, no tile's multiple
    a, sa = codes(min(M, period), K, g), scales_like(min(M, period), K, g)
    b, sb = codes(min(N, period), K, g), scales_like(blocks(min(N, period)), K, g)
    c = torch.zeros(M, N, dtype=torch.bfloat16, device="cuda")

    def wide(t, rows, p):
        if rows <= p:
            return t
        cols = t.shape[1]
        return repeated(rows, p, t.as_strided((t.shape[0], t.stride(0)), (t.stride(0), 1)).view(
            torch.uint8)).view(t.dtype)[:, :cols]

    qr.qr_gemm_f8(wide(a, M, period), wide(sa, M, period), wide(b, N, period), wide(sb, blocks(N), period // 128), c)
    want, tol = reference(a, sa, b, sb, None)
    for i in range(0, M, period * 16):
        for j in range(0, N, period * 16):
            part = c[i:i + period * 16, j:j + period * 16]
            again = (-(-part.shape[0] // want.shape[0]), -(-part.shape[1] // want.shape[1]))
            wide_want, wide_tol = (t.repeat(again)[:part.shape[0], :part.shape[1]] for t in (want, tol))
            check_product(part, wide_want, wide_tol, (M, N, K, i, j))


@pytest.mark.parametrize("N", [48, 1030])
def test_groups_beyond_4_gib(qr, N):  # noqa: F811
    """tokens read in place from a buffer of nearly 2^32 bytes, and its scales from another; weights of more"""
    K, E, M = 8192, 16, 2000
    tokens = ((1 << 32) - (1 << 18)) // K - 1
    ldsa = (((1 << 32) - (1 << 18)) // (4 * tokens) - 1) // 4 * 4
    assert tokens * K > (1 << 32) - (1 << 19) and 4 * tokens * ldsa > 1.99 * (1 << 31)
    say("grouped", tokens, N)
    g = torch.Generator(device="cuda").manual_seed(N)
    few, period = codes(1021, K, g), 1021
    a = repeated(tokens, period, few.view(torch.uint8)).view(F8)
    sa = torch.zeros(tokens, ldsa, device="cuda")[:, :K // 128]
    sa.copy_(repeated(tokens, 997, scales_like(997, K, g)))
    gap = ((1 << 32) // (E - 1) // K + 1) * K         # from one expert's weights to the next
    assert gap >= N * K and gap * (E - 1) > 1 << 32
    raw = torch.zeros(gap * (E - 1) + N * K, dtype=torch.uint8, device="cuda")
    b = raw.as_strided((E, N, K), (gap, K, 1)).view(F8)
    b.copy_(codes(E * N, K, g).unflatten(0, (E, N)))
    sb = scales_like(E * blocks(N), K, g).unflatten(0, (E, blocks(N)))
    offsets = (torch.arange(E + 1, device="cuda") * M // E).to(torch.int32)
    rows = torch.randint(0, tokens, (M,), generator=g, device="cuda").to(torch.int32)
    rows[:40], rows[-40:] = tokens - 1 - torch.arange(40, device="cuda", dtype=torch.int32), tokens - 1
    c = torch.zeros(M, N, dtype=torch.bfloat16, device="cuda")
    qr.qr_gemm_f8_grouped(a, sa, b, sb, offsets, c, rows=rows)
    ends = offsets.tolist()
    for e in range(E):
        at = rows[ends[e]:ends[e + 1]].long()
        x = a.view(torch.uint8)[at].view(F8)
        check_product(c[ends[e]:ends[e + 1]], *reference(x, sa[at], b[e].contiguous(), sb[e], None), (N, e))
