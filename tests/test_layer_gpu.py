"""The operators of include/qr_layer.h on the GPU against plain numpy in 64
bits (and, where every step is a single binary32 operation, bit for bit).

Tolerances, derived from the operations and fixed before the first run
(e = 2^-24, half a unit in the last place of binary32):
  h       one binary32 addition and one rounding to 16 bits, as numpy and
          torch do them: bit-exact;
  codes   of the norm: u = h*weight is exact, a = max|u| is exact, and the
          code is the exact quotient's: bit-exact.  In 64 bits 127*u is exact
          and the quotient rounded once; a tie stays one, and anything else
          is at least 2^-33 away from one (u and a have 24 bits);
  scale   of the norm: the sum of squares is a chain of at most CHAIN
          additions of positive terms (each within e), so r is within
          (CHAIN/2 + 4) e, and a*r/127 adds two roundings;
  silu    exp(-g): the exponent is rounded (|g| e), v_exp_f32 and v_rcp_f32
          are within one unit (2e each), 1+exp and the two products within e:
          v is within (|g| + 8) e of its value, and so is a; a code is within
          half a step plus 127 times twice that (and f, u*f: 4e) of
          127*v/a;
  product the integer sum is exact; its conversion, sa*sb, the product of
          the two and the sum with the bias are one rounding each, and the
          result is rounded once to 16 bits (half a step of the type)."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

E = 2.0 ** -24
TINY = 2.0 ** -119
TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def qr():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    from quantized_two_stage_amd import qr as q
    return q


def say(*a):
    print(*a, flush=True)


def chain(d):
    """additions a square passes through: within a lane, then across lanes"""
    per_lane = 32 if d <= 32768 else 8 * -(-d // 8192)
    return per_lane + 6 + 16


def rows_in(M, d, ld, dtype, fill, device="cuda"):
    """[M, d] inside a buffer filled with `fill`, the rows ld apart and one
    element off the buffer's start"""
    buf = torch.full((M * ld + 8,), fill, dtype=dtype, device=device)
    return buf, buf[1:1 + M * ld].view(M, ld)[:, :d]


def only_rows_written(buf, M, d, ld, fill):
    keep = torch.ones(buf.numel(), dtype=torch.bool, device=buf.device)
    keep[1:1 + M * ld].view(M, ld)[:, :d] = False
    return bool((buf[keep] == fill).all())


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def check_codes(q, s, u, r, tol_scale, label):
    """q, s of rows u (float64, exact in binary32) with factor r per row"""
    q, s = q.cpu().numpy(), s.cpu().to(torch.float64).numpy()
    for m in range(u.shape[0]):
        if not np.all(np.isfinite(u[m])) or not np.isfinite(r[m]):
            assert np.isnan(s[m]) and not q[m].any(), (label, m, "row is not finite")
            continue
        a = np.float32(np.max(np.abs(u[m])))
        if a < TINY:
            assert s[m] == 0 and not q[m].any(), (label, m, "zero row")
            continue
        want = np.rint(127.0 * u[m] / np.float64(a))
        assert np.array_equal(q[m], want.astype(np.int8)), (label, m, np.nonzero(q[m] != want))
        exact = float(a) * r[m] / 127
        assert abs(s[m] - exact) <= tol_scale * exact, (label, m, s[m], exact)


def norm_reference(h, w, eps):
    h, w = f64(h), f64(w)
    with np.errstate(all="ignore"):
        ss = np.sum(h * h, axis=1)
        r = 1.0 / np.sqrt(ss / h.shape[1] + eps)
        r[~np.isfinite(ss) | (ss > 3.4028235e38)] = np.nan
        return h * w, r


SHAPES = [(1, 8), (1, 1), (3, 7), (2, 9), (5, 64), (1, 8192), (4, 511), (3, 513), (7, 1000),
          (2, 2047), (3, 2048), (2, 2049), (2, 5003), (3, 8191), (2, 8200), (2, 16384),
          (1, 32767), (2, 32769), (1, 40000), (1, 131071), (300, 72), (259, 1040)]


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("M,d", SHAPES)
def test_norm(qr, M, d, dtype):
    t = TYPES[dtype]
    g = torch.Generator(device="cuda").manual_seed(M * 1000003 + d)
    randn = lambda *n: torch.randn(*n, generator=g, device="cuda")  # noqa: E731
    for kind in ("strided", "no residual", "in place"):
        say("norm", M, d, dtype, kind)
        ld = d + (0 if kind == "in place" else 5)
        _, x = rows_in(M, d, ld, t, 3.0)
        x.copy_(randn(M, d))
        w = (1 + 0.3 * randn(d)).to(t)
        hbuf, h = rows_in(M, d, ld, t, 3.0)
        qbuf, q = rows_in(M, d, d + 3, torch.int8, 77)
        s = torch.full((M,), 5.0, device="cuda")
        res = None
        if kind == "strided":
            res = (4 * randn(M, d)).to(t)
        elif kind == "in place":
            h.copy_(4 * randn(M, d))
            res = h
        want = (x.float() + res.float()).to(t) if res is not None else x.clone()
        qr.qr_add_rmsnorm_q8(x, res, w, 1e-5, h if res is not None else None, q, s)
        torch.cuda.synchronize()
        if res is not None:
            assert torch.equal(h, want)
            assert only_rows_written(hbuf, M, d, ld, 3.0)
        assert only_rows_written(qbuf, M, d, d + 3, 77)
        u, r = norm_reference(want, w, float(np.float32(1e-5)))
        check_codes(q, s, u, r, (chain(d) / 2 + 6) * E, (M, d, dtype, kind))


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("d", [5, 8, 72, 2500, 9000, 33000])
def test_norm_special_rows(qr, d, dtype):
    """zeros, one value, the type's largest and lowest values, subnormals,
    infinities and NaN in x, in the residual and in the weight"""
    t = TYPES[dtype]
    top, low = torch.finfo(t).max, torch.finfo(t).smallest_normal
    rows = []
    for k in range(10):
        x = torch.randn(d, device="cuda")
        if k == 0:
            x = torch.zeros(d, device="cuda")
        elif k == 1:
            x = torch.zeros(d, device="cuda")
            x[d - 1] = 0.5
        elif k == 2:
            x[d // 2] = float("inf")
        elif k == 3:
            x[0] = float("nan")
        elif k == 4:
            x[d - 1] = -float("inf")
        elif k == 5:
            x = torch.full((d,), -top, device="cuda")
        elif k == 6:
            x = torch.full((d,), low / 4, device="cuda")
        elif k == 7:
            x[d // 3] = top
        rows.append(x.to(t))
    x = torch.stack(rows)
    M = x.shape[0]
    res = torch.zeros_like(x)
    res[5] = -top                           # the sum overflows the type
    res[8, d - 1] = float("nan")
    for bad in (None, float("nan"), float("inf")):
        w = torch.ones(d, dtype=t, device="cuda")
        if bad is not None:
            w[d // 2] = bad
        h, (q, s) = torch.empty_like(x), qr.alloc_q8(M, d)
        qr.qr_add_rmsnorm_q8(x, res, w, 1e-6, h, q, s)
        torch.cuda.synchronize()
        want = (x.float() + res.float()).to(t)
        assert torch.equal(torch.nan_to_num(h, nan=1.0), torch.nan_to_num(want, nan=1.0))
        with np.errstate(invalid="ignore"):
            u, r = norm_reference(want, w, float(np.float32(1e-6)))
        check_codes(q, s, u, r, (chain(d) / 2 + 6) * E, (d, dtype, bad))


def test_norm_far_rows(qr):
    """row offsets past 2^32 bytes"""
    M, d, ld = 40000, 64, 65536
    buf = torch.empty(M * ld, dtype=torch.bfloat16, device="cuda")
    x = buf.view(M, ld)[:, 100:100 + d]
    x.copy_(torch.randn(M, d, device="cuda"))
    w = torch.ones(d, dtype=torch.bfloat16, device="cuda")
    q, s = qr.alloc_q8(M, d)
    qr.qr_add_rmsnorm_q8(x, None, w, 1e-5, None, q, s)
    torch.cuda.synchronize()
    at = [0, 1, 32767, 32768, 39998, 39999]
    u, r = norm_reference(x[at], w, float(np.float32(1e-5)))
    check_codes(q[at], s[at], u, r, (chain(d) / 2 + 6) * E, "far rows")


GATHER_SHAPES = [(1, 8), (3, 8), (2, 40), (5, 64), (7, 72), (1, 2048), (3, 2056), (2, 8192),
                 (3, 8200), (1, 32776), (33, 264)]


@pytest.mark.parametrize("dtype", [0, 1, 2])
@pytest.mark.parametrize("codec", [0, 5, 1, 2, 3, 9, 10, 11])
def test_gather_norm(qr, codec, dtype):
    """bit for bit what qr_dequantize and qr_add_rmsnorm_q8 give, with and
    without a residual; the first wire image is quantized values, the second
    arbitrary bytes (scales and zeros of any value, NaN among them)"""
    t = torch.float16 if dtype == 0 else torch.bfloat16
    for M, d in GATHER_SHAPES:
        n = M * d
        g = torch.Generator(device="cuda").manual_seed(n + 17 * codec + dtype)
        for kind in ("quantized", "bytes"):
            say("gather", codec, dtype, M, d, kind)
            wire = qr.alloc_wire(codec, n)
            if kind == "quantized":
                x = torch.randn(n, generator=g, device="cuda").to(t)
                qr.qr_quantize(codec, x, wire, dtype=dtype)
            else:
                wire.copy_(torch.randint(0, 256, wire.shape, generator=g, device="cuda"))
            w = (1 + 0.3 * torch.randn(d, generator=g, device="cuda")).to(t)
            x = torch.empty(M, d, dtype=t, device="cuda")
            qr.qr_dequantize(codec, wire, x, dtype=dtype)
            for res in (None, (4 * torch.randn(M, d, generator=g, device="cuda")).to(t)):
                hbuf, h = rows_in(M, d, d + 7, t, 3.0)
                q, s = qr.alloc_q8(M, d)
                qr.qr_gather_add_rmsnorm_q8(codec, wire, res, w, 1e-5, h, q, s, dtype=dtype)
                q2, s2 = qr.alloc_q8(M, d)
                h2 = torch.empty_like(x) if res is not None else None
                qr.qr_add_rmsnorm_q8(x, res, w, 1e-5, h2, q2, s2)
                torch.cuda.synchronize()
                h2 = x if h2 is None else h2
                assert torch.equal(torch.isnan(h), torch.isnan(h2))
                assert torch.equal(torch.nan_to_num(h).view(torch.int16),
                                   torch.nan_to_num(h2).view(torch.int16))
                assert torch.equal(q, q2) and torch.equal(s.isnan(), s2.isnan())
                assert torch.equal(torch.nan_to_num(s), torch.nan_to_num(s2))
                assert only_rows_written(hbuf, M, d, d + 7, 3.0)


@pytest.mark.parametrize("codec", [0, 5, 1, 2, 3, 9, 10, 11])
def test_gather_norm_against_the_oracle(qr, codec):
    """the wire decoded by the scalar C reference, the rest in 64 bits"""
    import oracle
    M, d = 6, 1032
    x = torch.randn(M * d, device="cuda", generator=torch.Generator("cuda").manual_seed(codec))
    x = x.to(torch.float16)
    wire = qr.alloc_wire(codec, M * d)
    qr.qr_quantize(codec, x, wire)
    want = oracle.dequantize(codec, 0, wire.cpu().numpy(), M * d)
    want = torch.from_numpy(want.view(np.float16).reshape(M, d).copy()).cuda()
    w = (1 + 0.3 * torch.randn(d, device="cuda")).to(torch.float16)
    h = torch.empty(M, d, dtype=torch.float16, device="cuda")
    q, s = qr.alloc_q8(M, d)
    qr.qr_gather_add_rmsnorm_q8(codec, wire, None, w, 1e-5, h, q, s)
    torch.cuda.synchronize()
    assert torch.equal(h.view(torch.int16), want.view(torch.int16))
    u, r = norm_reference(want, w, float(np.float32(1e-5)))
    check_codes(q, s, u, r, (chain(d) / 2 + 6) * E, codec)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("M,d", [(1, 1), (2, 7), (3, 8), (1, 4096), (5, 33), (4, 513), (3, 2051),
                                 (2, 8193), (2, 16384), (1, 32771), (1, 131071), (270, 96)])
def test_silu(qr, M, d, dtype):
    t = TYPES[dtype]
    g = torch.Generator(device="cuda").manual_seed(M * 7919 + d)
    say("silu", M, d, dtype)
    _, gu = rows_in(M, 2 * d, 2 * d + 3, t, 3.0)
    gu.copy_(2 * torch.randn(M, 2 * d, generator=g, device="cuda"))
    qbuf, q = rows_in(M, d, d + 5, torch.int8, 77)
    s = torch.full((M,), 5.0, device="cuda")
    qr.qr_silu_mul_q8(gu, q, s)
    torch.cuda.synchronize()
    assert only_rows_written(qbuf, M, d, d + 5, 77)
    check_silu(gu, q, s, (M, d, dtype))


def check_silu(gu, q, s, label):
    x, q, s = f64(gu), q.cpu().numpy().astype(np.float64), s.cpu().to(torch.float64).numpy()
    d = x.shape[1] // 2
    with np.errstate(all="ignore"):
        v = x[:, :d] / (1 + np.exp(-x[:, :d])) * x[:, d:]
    for m in range(x.shape[0]):
        if not np.all(np.isfinite(x[m])):
            assert np.isnan(s[m]) and not q[m].any(), (label, m)
            continue
        a = np.max(np.abs(v[m]))
        if a == 0:
            assert s[m] == 0 and not q[m].any(), (label, m)
            continue
        off = (np.max(np.abs(x[m, :d])) + 8) * E
        assert abs(s[m] * 127 - a) <= (off + 2 * E) * a, (label, m)
        assert np.max(np.abs(q[m] - 127 * v[m] / a)) <= 0.5 + 127 * (2 * off + 4 * E), (label, m)
        assert np.max(np.abs(q[m])) == 127, (label, m)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("d", [3, 64, 3000, 20000])
def test_silu_special_rows(qr, d, dtype):
    """zeros, large gates of both signs, infinities and NaN in either half"""
    t = TYPES[dtype]
    gu = torch.randn(9, 2 * d, device="cuda").to(t)
    gu[0] = 0
    gu[1, :d] = 0
    gu[2, 0] = 80.0
    gu[2, 1] = -80.0
    gu[3, d - 1] = float("nan")
    gu[4, 2 * d - 1] = float("inf")
    gu[5, 1] = float("inf")
    gu[6, 0] = -float("inf")
    gu[7, :d] = 200.0
    gu[7, 1] = -200.0
    q, s = qr.alloc_q8(9, d)
    qr.qr_silu_mul_q8(gu, q, s)
    torch.cuda.synchronize()
    check_silu(gu, q, s, (d, dtype))


# --------------------------------------------------------------------------- products


def codes_in(rows, K, g, ld=None, amp=256):
    """[rows, K] codes whose padding up to the next multiple of 16 (and the
    rest of the stride) holds other codes"""
    ld = -(-K // 16) * 16 if ld is None else ld
    return torch.randint(-amp // 2, amp // 2, (rows, ld), generator=g, device="cuda",
                         dtype=torch.int8)[:, :K]


def check_product(qr, M, N, K, t, bias, g, lda=None, ldb=None, amp=256, pad=3):
    a, b = codes_in(M, K, g, lda, amp), codes_in(N, K, g, ldb, amp)
    sa = torch.rand(M, generator=g, device="cuda") * 0.02 + 0.001
    sb = (torch.rand(N, generator=g, device="cuda") + 0.1) / (16 * K ** 0.5)
    bv = torch.randn(N, generator=g, device="cuda").to(t) if bias else None
    cbuf, c = rows_in(M, N, N + pad, t, 3.0)
    ws = qr.alloc_gemm_workspace(M, N, K)
    if ws is not None:
        ws.fill_(0xA7)
    qr.qr_gemm_i8(a, sa, b, sb, c, bias=bv, workspace=ws)
    torch.cuda.synchronize()
    assert only_rows_written(cbuf, M, N, N + pad, 3.0)
    # exact: below 2^53 in every partial sum
    exact = (a.double() @ b.double().t()).cpu().numpy()
    scale = f64(sa)[:, None] * f64(sb)[None, :]
    off = f64(bv)[None, :] if bias else 0.0
    want = exact * scale + off
    size = np.abs(exact * scale)
    slack = (3 * size + np.abs(want) + np.abs(off)) * E * 1.01
    half = np.abs(want) * torch.finfo(t).eps / 2 + torch.finfo(t).smallest_normal * \
        torch.finfo(t).eps / 2
    err = np.abs(f64(c) - want)
    bad = err > slack * (1 + torch.finfo(t).eps) + half
    assert not bad.any(), (M, N, K, t, np.argwhere(bad)[:4], f64(c)[bad][:4], want[bad][:4])


GEMM_SHAPES = [
    (1, 1, 1), (1, 5, 15), (1, 64, 16), (1, 130, 17), (1, 1000, 64), (1, 4099, 2050),
    (1, 8192, 8192), (2, 33, 63), (3, 255, 65), (4, 512, 4096), (5, 16, 16384), (8, 300, 127),
    (9, 1024, 1024), (15, 77, 128), (16, 256, 129), (16, 2048, 4096), (17, 64, 1000),
    (31, 129, 255), (32, 4096, 512), (33, 100, 333), (48, 1000, 2050), (63, 513, 640),
    (64, 64, 64), (64, 1024, 8192), (65, 65, 65), (96, 250, 1500), (127, 255, 257),
    (128, 128, 128), (128, 2048, 2048), (129, 257, 1025), (200, 700, 300), (255, 256, 256),
    (256, 256, 8192), (257, 511, 384), (300, 1000, 96), (333, 5003, 2050), (512, 512, 512),
    (700, 1300, 31), (1000, 2000, 4000), (1024, 2048, 1040), (2049, 300, 272), (2048, 2304, 1024),
]


@pytest.mark.parametrize("M,N,K", GEMM_SHAPES)
def test_gemm(qr, M, N, K):
    g = torch.Generator(device="cuda").manual_seed(M * 31 + N * 17 + K)
    for t in (torch.float16, torch.bfloat16):
        for bias in (False, True):
            say("gemm", M, N, K, t, bias)
            check_product(qr, M, N, K, t, bias, g, pad=3 if bias else 0)


def test_gemm_random_shapes(qr):
    r = np.random.RandomState(11)
    g = torch.Generator(device="cuda").manual_seed(12)
    for i in range(120):
        M, N, K = (int(round(2 ** r.uniform(0, top))) for top in (11, 11.5, 12.5))
        if r.rand() < 0.4:
            M, N, K = max(1, M // 16 * 16), max(1, N // 64 * 64), max(1, K // 128 * 128)
        say("gemm", i, M, N, K)
        pads = [16 * int(r.randint(0, 9)) for _ in range(2)]
        check_product(qr, M, N, K, (torch.float16, torch.bfloat16)[i % 2], bool(i % 3), g,
                      lda=-(-K // 16) * 16 + pads[0], ldb=-(-K // 16) * 16 + pads[1],
                      pad=int(r.randint(0, 9)))


@pytest.mark.parametrize("M,N", [(1, 40), (7, 300), (40, 70), (130, 260)])
def test_gemm_largest_sums(qr, M, N):
    """K at its limit with every code -128 (the largest sum, 2^31 - 16384),
    and with 127 against -128"""
    K, ld = 131071, 131072
    for x, y in ((-128, -128), (127, -128)):
        a = torch.full((M, ld), x, dtype=torch.int8, device="cuda")[:, :K]
        b = torch.full((N, ld), y, dtype=torch.int8, device="cuda")[:, :K]
        sa, sb = torch.full((M,), 2.0 ** -20, device="cuda"), torch.ones(N, device="cuda")
        c = torch.empty(M, N, dtype=torch.float16, device="cuda")
        qr.qr_gemm_i8(a, sa, b, sb, c, workspace=qr.alloc_gemm_workspace(M, N, K))
        torch.cuda.synchronize()
        want = torch.tensor(np.float32(x * y * K) * np.float32(2.0 ** -20)).to(torch.float16)
        assert bool((c == want.cuda()).all()), (x, y, c[0, 0], want)


@pytest.mark.parametrize("M", [1, 20, 200])
def test_gemm_rows_without_a_scale(qr, M):
    """a token or a channel whose scale is NaN gives NaN in its row or column
    and nowhere else; a scale of 0 gives the bias"""
    N, K = 200, 300
    g = torch.Generator(device="cuda").manual_seed(5)
    a, b = codes_in(M, K, g), codes_in(N, K, g)
    sa, sb = torch.ones(M, device="cuda"), torch.full((N,), 0.01, device="cuda")
    sa[M - 1], sb[7] = float("nan"), float("nan")
    if M > 1:
        sa[0] = 0.0
    bias = torch.arange(N, device="cuda").to(torch.bfloat16)
    c = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    qr.qr_gemm_i8(a, sa, b, sb, c, bias=bias, workspace=qr.alloc_gemm_workspace(M, N, K))
    torch.cuda.synchronize()
    nan = torch.zeros(M, N, dtype=torch.bool, device="cuda")
    nan[M - 1], nan[:, 7] = True, True
    assert torch.equal(c.isnan(), nan)
    if M > 1:
        keep = torch.arange(N, device="cuda") != 7
        assert torch.equal(c[0][keep], bias[keep])


@pytest.mark.parametrize("M", [3, 700])
def test_gemm_far_rows(qr, M):
    """row offsets past 2^31 bytes in a, b and c"""
    N, K, ld = 700, 200, (1 << 23) - 16
    a = torch.zeros(M, ld, dtype=torch.int8, device="cuda")[:, 4096:4096 + K]
    b = torch.zeros(N, ld, dtype=torch.int8, device="cuda")[:, 4096:4096 + K]
    g = torch.Generator(device="cuda").manual_seed(M)
    a.copy_(codes_in(M, K, g))
    b.copy_(codes_in(N, K, g))
    sa, sb = torch.ones(M, device="cuda"), torch.ones(N, device="cuda") * 2.0 ** -10
    c = torch.empty(M, 4000000, dtype=torch.bfloat16, device="cuda")[:, :N]
    qr.qr_gemm_i8(a, sa, b, sb, c, workspace=qr.alloc_gemm_workspace(M, N, K))
    torch.cuda.synchronize()
    want = ((a.double() @ b.double().t()).float() * 2.0 ** -10).to(torch.bfloat16)
    assert torch.equal(c, want)


def test_results_do_not_depend_on_the_run(qr):
    """the same call twice gives the same bits"""
    g = torch.Generator(device="cuda").manual_seed(3)
    for M, N, K in ((1, 4096, 8192), (48, 1024, 8192), (300, 2000, 4096)):
        a, b = codes_in(M, K, g), codes_in(N, K, g)
        sa, sb = torch.rand(M, device="cuda"), torch.rand(N, device="cuda")
        ws = qr.alloc_gemm_workspace(M, N, K)
        c = [torch.empty(M, N, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        for x in c:
            qr.qr_gemm_i8(a, sa, b, sb, x, workspace=ws)
        torch.cuda.synchronize()
        assert torch.equal(c[0].view(torch.int16), c[1].view(torch.int16))


# --------------------------------------------------------------------------- streams, graphs


def _chain(qr, t, M, d, f):
    """one rank's share of a layer's feed-forward part: its buffers and calls"""
    g = torch.Generator(device="cuda").manual_seed(M + d)
    randn = lambda *n: torch.randn(*n, generator=g, device="cuda")  # noqa: E731
    n = M * d
    x = randn(n).to(t)
    wire = qr.alloc_wire(qr.QR_Q6, n)
    qr.qr_quantize(qr.QR_Q6, x, wire)
    res, w = (3 * randn(M, d)).to(t), (1 + 0.2 * randn(d)).to(t)
    b1, b2 = codes_in(2 * f, d, g), codes_in(d, f, g)
    s1, s2 = torch.rand(2 * f, device="cuda") * 1e-3, torch.rand(d, device="cuda") * 1e-3
    h, (q, s) = torch.empty(M, d, dtype=t, device="cuda"), qr.alloc_q8(M, d)
    gu, (qa, ss) = torch.empty(M, 2 * f, dtype=t, device="cuda"), qr.alloc_q8(M, f)
    y = torch.empty(M, d, dtype=t, device="cuda")
    w1, w2 = qr.alloc_gemm_workspace(M, 2 * f, d), qr.alloc_gemm_workspace(M, d, f)

    def run(stream=None):
        qr.qr_gather_add_rmsnorm_q8(qr.QR_Q6, wire, res, w, 1e-5, h, q, s, stream=stream)
        qr.qr_gemm_i8(q, s, b1, s1, gu, workspace=w1, stream=stream)
        qr.qr_silu_mul_q8(gu, qa, ss, stream=stream)
        qr.qr_gemm_i8(qa, ss, b2, s2, y, workspace=w2, stream=stream)
    return run, (h, q, s, gu, qa, ss, y), (wire, res)


@pytest.mark.parametrize("M,d,f", [(1, 1024, 520), (40, 512, 1000), (300, 1024, 512)])
def test_other_streams_and_graphs(qr, M, d, f):
    run, outs, ins = _chain(qr, torch.bfloat16, M, d, f)
    run()
    torch.cuda.synchronize()
    want = [o.clone() for o in outs]
    # another stream, by argument and as the current one
    side = torch.cuda.Stream()
    for how in ("argument", "current"):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        if how == "argument":
            run(stream=side)
        else:
            with torch.cuda.stream(side):
                run()
        side.synchronize()
        for o, x in zip(outs, want):
            assert torch.equal(o, x), how
    # a graph replays what the eager calls give, with eager work between
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for k in range(4):
        ins[1].mul_(0.5 if k % 2 else 1.5)
        run()
        torch.cuda.synchronize()
        want = [o.clone() for o in outs]
        for o in outs:
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for o, x in zip(outs, want):
            assert torch.equal(o, x), k


def test_refusals_write_nothing(qr):
    M, d = 4, 64
    x = torch.randn(M, d, device="cuda").half()
    w = torch.ones(d, dtype=torch.float16, device="cuda")
    h = torch.full_like(x, 3.0)
    q, s = torch.full((M, d), 7, dtype=torch.int8, device="cuda"), torch.full((M,), 9.0,
                                                                              device="cuda")
    with pytest.raises(qr.QRError, match="eps"):
        qr.qr_add_rmsnorm_q8(x, x.clone(), w, 0.0, h, q, s)
    with pytest.raises(qr.QRError, match="together"):
        qr.qr_add_rmsnorm_q8(x, None, w, 1e-5, h, q, s)
    with pytest.raises(ValueError, match="shape"):
        qr.qr_add_rmsnorm_q8(x, x[:, :32], w, 1e-5, h, q, s)
    with pytest.raises(TypeError, match="bfloat16"):
        qr.qr_add_rmsnorm_q8(x, x.bfloat16(), w, 1e-5, h, q, s)
    with pytest.raises(ValueError, match="not on GPU"):
        qr.qr_add_rmsnorm_q8(x, x.clone(), w.cpu(), 1e-5, h, q, s)
    with pytest.raises(qr.QRError, match="stride"):
        qr.qr_silu_mul_q8(x[:1].expand(M, d), q[:, :32], s)
    with pytest.raises(ValueError, match="wire holds"):
        qr.qr_gather_add_rmsnorm_q8(qr.QR_Q8, q.reshape(-1)[:128], None, w, 1e-5, h, q, s)
    with pytest.raises(qr.QRError, match="multiple of 16"):
        qr.qr_gemm_i8(torch.zeros(4, 72, dtype=torch.int8, device="cuda")[:, :64], s, q, s,
                      torch.zeros(4, 4, dtype=torch.float16, device="cuda"))
    torch.cuda.synchronize()
    assert bool((h == 3).all()) and bool((q == 7).all()) and bool((s == 9).all())


def test_no_tokens(qr):
    w = torch.ones(64, dtype=torch.float16, device="cuda")
    x = torch.empty(0, 64, dtype=torch.float16, device="cuda")
    q, s = qr.alloc_q8(0, 64)
    qr.qr_add_rmsnorm_q8(x, x.clone(), w, 1e-5, x.clone(), q, s)
    qr.qr_gather_add_rmsnorm_q8(qr.QR_Q8, torch.empty(0, dtype=torch.uint8, device="cuda"), x, w,
                                1e-5, x.clone(), q, s)
    qr.qr_silu_mul_q8(torch.empty(0, 128, dtype=torch.float16, device="cuda"), q, s)
    b, sb = qr.alloc_q8(8, 64)
    c = torch.empty(0, 8, dtype=torch.float16, device="cuda")
    assert qr.qr_gemm_i8(q, s, b, sb, c).shape == (0, 8)
