"""The operators of include/qr_f8.h on the host (no GPU needed): the library exports and binds every declared function,
and every invalid argument is rejected with its documented code before anything is launched (the pointers below are
fake, never touched); the binding rejects what only the tensors know."""
import os
import re

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "qr_f8.h")
FAKE = 0x7f0000000000
MB = 1 << 20
NAN, INF = float("nan"), float("inf")
F8 = torch.float8_e4m3fn
ARG, UNSUPPORTED, SIZE, ALIGN, WORKSPACE = -1, -2, -3, -4, -5


def _qr():
    from quantized_two_stage_amd import qr
    return qr


def test_every_declared_function_is_exported_and_bound():
    qr = _qr()
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(qr_[a-z0-9_]+)\s*\(", src)))
    assert names == ["qr_add_rmsnorm_f8", "qr_combine", "qr_gemm_f8", "qr_gemm_f8_grouped", "qr_route",
                     "qr_route_workspace_bytes", "qr_silu_mul_f8"]
    for name in names:
        assert hasattr(qr.LIB, name) and name in qr.EXPORTS and callable(getattr(qr, name))


def at(n):
    return FAKE + n * MB


def _norm(dtype=1, x=FAKE, ldx=300, res=at(1), ldr=300, w=at(2), eps=1e-5, M=4, d=300, h=at(3), ldh=300, y=at(4),
          ldy=300, q=at(5), ldq=300, s=at(6), lds=3):
    return _qr().LIB.qr_add_rmsnorm_f8(dtype, x, ldx, res, ldr, w, eps, M, d, h, ldh, y, ldy, q, ldq, s, lds, None)


def _silu(dtype=1, gu=FAKE, ldg=600, M=4, d=300, q=at(1), ldq=300, s=at(2), lds=3):
    return _qr().LIB.qr_silu_mul_f8(dtype, gu, ldg, M, d, q, ldq, s, lds, None)


def _gemm(dtype=1, a=FAKE, lda=304, sa=at(1), ldsa=4, b=at(2), ldb=304, sb=at(3), ldsb=3, bias=None, M=4, N=200, K=300,
          c=at(4), ldc=200):
    return _qr().LIB.qr_gemm_f8(dtype, a, lda, sa, ldsa, b, ldb, sb, ldsb, bias, M, N, K, c, ldc, None)


def _grouped(dtype=1, a=FAKE, lda=304, sa=at(1), ldsa=4, rows=at(5), tokens=3, b=at(2), ldb=304, gb=304 * 200, sb=at(3),
             ldsb=3, gsb=6, bias=None, ldbias=200, off=at(6), E=5, M=4, N=200, K=300, c=at(7), ldc=200):
    return _qr().LIB.qr_gemm_f8_grouped(dtype, a, lda, sa, ldsa, rows, tokens, b, ldb, gb, sb, ldsb, gsb, bias, ldbias,
                                        off, E, M, N, K, c, ldc, None)


def _route(dtype=1, x=FAKE, ldl=16, T=100, E=16, k=4, renorm=0, w=at(1), e=at(2), o=at(3), r=at(4), p=at(5), ws=at(6),
           ws_bytes=None):
    qr = _qr()
    need = qr.qr_route_workspace_bytes(T, E, k) if ws_bytes is None else ws_bytes
    return qr.LIB.qr_route(dtype, x, ldl, T, E, k, renorm, w, e, o, r, p, ws, need, None)


def _combine(dtype=1, c=FAKE, ldc=64, R=8, p=at(1), w=at(2), T=4, k=2, d=64, add=at(3), lda=64, y=at(4), ldy=64):
    return _qr().LIB.qr_combine(dtype, c, ldc, R, p, w, T, k, d, add, lda, y, ldy, None)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), UNSUPPORTED), (dict(dtype=-1), UNSUPPORTED), (dict(d=0), SIZE), (dict(d=131072), SIZE),
    (dict(M=(1 << 22) + 1), SIZE), (dict(x=None), ARG), (dict(w=None), ARG), (dict(q=None), ARG), (dict(s=None), ARG),
    (dict(res=None), ARG), (dict(h=None), ARG), (dict(eps=0.0), ARG), (dict(eps=NAN), ARG), (dict(eps=INF), ARG),
    (dict(ldx=299), ARG), (dict(ldr=299), ARG), (dict(ldh=1), ARG), (dict(ldy=299), ARG), (dict(ldq=299), ARG),
    (dict(lds=2), ARG), (dict(x=FAKE + 1), ALIGN), (dict(y=at(4) + 1), ALIGN), (dict(s=at(6) + 2), ALIGN),
    (dict(h=FAKE + 64), ARG), (dict(h=at(1) + 2), ARG), (dict(h=at(1), ldh=304), ARG), (dict(y=FAKE), ARG),
    (dict(y=at(1)), ARG), (dict(y=at(3)), ARG), (dict(y=at(2)), ARG), (dict(q=at(4)), ARG), (dict(q=at(6)), ARG),
    (dict(s=at(4) + 600), ARG), (dict(q=FAKE), ARG), (dict(s=at(2)), ARG), (dict(s=at(5) + 1196), ARG),
])
def test_norm_rejects(kw, code):
    assert _norm(**kw) == code
    assert _qr().qr_last_error() != ""


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), UNSUPPORTED), (dict(d=0), SIZE), (dict(M=(1 << 22) + 1), SIZE), (dict(gu=None), ARG),
    (dict(q=None), ARG), (dict(s=None), ARG), (dict(ldg=599), ARG), (dict(ldq=299), ARG), (dict(lds=2), ARG),
    (dict(gu=FAKE + 1), ALIGN), (dict(s=at(2) + 1), ALIGN), (dict(q=FAKE + 600), ARG), (dict(s=FAKE), ARG),
    (dict(s=at(1) + 4), ARG),
])
def test_silu_rejects(kw, code):
    assert _silu(**kw) == code
    assert _qr().qr_last_error() != ""


PRODUCT = [
    (dict(dtype=2), UNSUPPORTED), (dict(K=0), SIZE), (dict(N=0), SIZE), (dict(K=131072), SIZE),
    (dict(N=(1 << 22) + 1), SIZE), (dict(M=(1 << 22) + 1), SIZE), (dict(a=None), ARG), (dict(sa=None), ARG),
    (dict(b=None), ARG), (dict(sb=None), ARG), (dict(c=None), ARG), (dict(lda=288), ARG), (dict(ldb=288), ARG),
    (dict(ldc=199), ARG), (dict(ldsa=2), ARG), (dict(ldsb=2), ARG), (dict(lda=312), ALIGN), (dict(ldb=312), ALIGN),
    (dict(ldsa=6), ALIGN), (dict(lda=1 << 23), SIZE), (dict(ldb=1 << 23), SIZE), (dict(ldsa=(1 << 20) + 4), SIZE),
    (dict(a=FAKE + 8), ALIGN), (dict(sa=at(1) + 4), ALIGN), (dict(b=at(2) + 8), ALIGN), (dict(sb=at(3) + 2), ALIGN),
    (dict(c=FAKE), ARG), (dict(c=at(1)), ARG), (dict(c=at(2) + 16), ARG), (dict(c=at(3)), ARG),
]


@pytest.mark.parametrize("kw,code", PRODUCT + [
    (dict(c=at(4) + 1), ALIGN), (dict(bias=at(5) + 1), ALIGN), (dict(bias=at(4)), ARG)])
def test_gemm_rejects(kw, code):
    assert _gemm(**kw) == code
    assert _qr().qr_last_error() != ""


@pytest.mark.parametrize("kw,code", PRODUCT + [
    (dict(E=0), SIZE), (dict(E=1025), SIZE), (dict(tokens=0), SIZE), (dict(tokens=(1 << 22) + 1), SIZE),
    (dict(off=None), ARG), (dict(off=at(6) + 2), ALIGN), (dict(rows=at(5) + 2), ALIGN), (dict(gb=304 * 200 + 8), ALIGN),
    (dict(gb=304 * 199), ARG), (dict(gsb=5), ARG), (dict(bias=at(8), ldbias=199), ARG), (dict(bias=at(8) + 1), ALIGN),
    (dict(bias=at(7)), ARG), (dict(c=at(6)), ARG), (dict(c=at(5)), ARG), (dict(c=at(2) + 304 * 200 * 4), ARG),
    (dict(tokens=1 << 20, lda=4096, b=1 << 50, sb=1 << 51, c=1 << 52, sa=1 << 49), SIZE),
    (dict(tokens=1 << 22, lda=304, ldsa=256, b=1 << 50, sb=1 << 51, c=1 << 52, sa=1 << 49), SIZE),
    # more tiles than a launch holds
    (dict(E=1024, M=1024, rows=None, K=16, lda=16, N=1 << 22, ldb=16, gb=1 << 26, gsb=3 << 15, ldc=1 << 22, sa=1 << 49,
          b=1 << 50, sb=1 << 51, c=1 << 52), SIZE),
])
def test_grouped_rejects(kw, code):
    assert _grouped(**kw) == code
    assert _qr().qr_last_error() != ""


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), UNSUPPORTED), (dict(dtype=4), UNSUPPORTED), (dict(E=0), SIZE), (dict(E=1025), SIZE), (dict(k=0), SIZE),
    (dict(k=17), SIZE), (dict(E=64, k=33, ldl=64), SIZE), (dict(T=(1 << 22) + 1, k=1), SIZE), (dict(T=1 << 21, k=4), SIZE),
    (dict(x=None), ARG), (dict(w=None), ARG), (dict(e=None), ARG), (dict(o=None), ARG), (dict(r=None), ARG),
    (dict(p=None), ARG), (dict(ldl=15), ARG), (dict(x=FAKE + 1), ALIGN), (dict(dtype=3, x=FAKE + 2), ALIGN),
    (dict(w=at(1) + 2), ALIGN), (dict(p=at(5) + 1), ALIGN), (dict(ws=None), ARG), (dict(ws=at(6) + 8), ALIGN),
    (dict(ws_bytes=16 * 2 * 2 - 1), WORKSPACE), (dict(ws=at(1)), ARG), (dict(ws=FAKE), ARG), (dict(w=FAKE), ARG),
    (dict(e=at(1)), ARG), (dict(o=at(2) + 4), ARG), (dict(r=at(3)), ARG), (dict(p=at(4)), ARG), (dict(p=FAKE), ARG),
])
def test_route_rejects(kw, code):
    assert _route(**kw) == code
    assert _qr().qr_last_error() != ""


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), UNSUPPORTED), (dict(dtype=3), UNSUPPORTED), (dict(d=0), SIZE), (dict(d=131072), SIZE),
    (dict(k=0), SIZE), (dict(k=33), SIZE), (dict(T=(1 << 22) + 1), SIZE), (dict(R=0), SIZE), (dict(R=(1 << 22) + 1), SIZE),
    (dict(c=None), ARG), (dict(p=None), ARG), (dict(w=None), ARG), (dict(y=None), ARG), (dict(ldc=63), ARG),
    (dict(lda=63), ARG), (dict(ldy=63), ARG), (dict(c=FAKE + 1), ALIGN), (dict(p=at(1) + 2), ALIGN),
    (dict(w=at(2) + 1), ALIGN), (dict(add=at(3) + 1), ALIGN), (dict(y=FAKE + 16), ARG), (dict(y=at(1)), ARG),
    (dict(y=at(2)), ARG), (dict(y=at(3) + 2), ARG), (dict(y=at(3), ldy=72), ARG),
])
def test_combine_rejects(kw, code):
    assert _combine(**kw) == code
    assert _qr().qr_last_error() != ""


def test_a_batch_without_tokens_is_nothing_to_do():
    qr = _qr()
    none = dict(x=None, res=None, h=None, y=None, q=None, s=None, w=None)
    assert _norm(M=0, **none) == 0 and _silu(M=0, gu=None, q=None, s=None) == 0
    assert _gemm(M=0, a=None, sa=None, c=None) == 0
    assert _grouped(M=0, tokens=0, a=None, sa=None, c=None, rows=None) == 0
    assert _combine(T=0, R=0, c=None, p=None, w=None, y=None) == 0
    assert qr.qr_last_error() == ""
    assert _norm(M=0, d=0) == SIZE and _gemm(M=0, K=0) == SIZE and _combine(T=0, k=0) == SIZE
    assert _route(T=0, o=None) == ARG


def test_route_workspace():
    qr = _qr()
    f = qr.qr_route_workspace_bytes
    assert f(1, 64, 8) == f(64, 1024, 8) == f(0, 8, 1) == 0
    assert f(65, 100, 8) == 2 * 104 * 2 and f(16384, 256, 8) == 256 * 256 * 2
    for T in (65, 16385, 70000, 1 << 22):
        assert 0 < f(T, 1024, 1) <= 256 * 1024 * 2
    assert f(100, 0, 1) == f(100, 2000, 1) == f(100, 8, 0) == f(1 << 23, 8, 1) == 0
    assert qr.alloc_route_workspace(64, 64, 8, device="cpu") is None
    assert qr.alloc_route_workspace(65, 64, 8, device="cpu").numel() == 256


def test_binding_rejects_tensors():
    """everything here is refused before a GPU would be needed"""
    qr = _qr()
    x, w = torch.zeros(2, 16).half(), torch.zeros(16).half()
    q, s = qr.alloc_f8(2, 16, device="cpu")
    with pytest.raises(ValueError, match="not on the current GPU"):
        qr.qr_add_rmsnorm_f8(x, x.clone(), w, 1e-5, x.clone(), None, q, s)
    with pytest.raises(TypeError, match="float16 or bfloat16"):
        qr.qr_add_rmsnorm_f8(x.float(), x, w, 1e-5, x, None, q, s)
    with pytest.raises(ValueError, match="differ in length"):
        qr.qr_silu_mul_f8(torch.zeros(2, 15).half(), q, s)
    with pytest.raises(TypeError, match="float16 or bfloat16"):
        qr.qr_gemm_f8(q, s, q, s, torch.zeros(2, 2))
    with pytest.raises(ValueError, match="not on the current GPU"):
        qr.qr_gemm_f8(q, s, q, s, x)
    with pytest.raises(ValueError, match="not on the current GPU"):
        qr.qr_gemm_f8_grouped(q, s, q[None], s[None], torch.zeros(2, dtype=torch.int32), x)
    with pytest.raises(TypeError, match="float32 expected"):
        qr.qr_route(torch.zeros(2, 4).double(), s, s, s, s, s)
    with pytest.raises(ValueError, match="not on the current GPU"):
        qr.qr_combine(x, s, s, x)
    # the checks of single arguments (device -1: tensors in host memory)
    with pytest.raises(TypeError, match="float8"):
        qr._pieces("a", torch.zeros(2, 16, dtype=torch.int8), 2, 16, F8, -1, 16)
    wide, scales = qr.alloc_f8(3, 300, device="cpu")
    assert wide.shape == (3, 300) and wide.stride() == (304, 1) and scales.shape == (3, 3) and scales.stride() == (4, 1)
    assert qr._pieces("a", wide, 3, 300, F8, -1, 16) == 304 and qr._pieces("sa", scales, 3, 3, torch.float32, -1, 4) == 4
    with pytest.raises(ValueError, match="padding"):
        qr._pieces("a", torch.zeros(1, 17).to(F8), 1, 17, F8, -1, 16)
    with pytest.raises(ValueError, match="padding"):
        qr._pieces("sa", torch.zeros(7).as_strided((2, 3), (4, 1)), 2, 3, torch.float32, -1, 4)
