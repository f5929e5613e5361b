"""The operators of include/qr_layer.h on the host (no GPU needed): the library
exports and binds every declared function, and every invalid argument is
rejected with its documented code before anything is launched (the pointers
below are fake, never touched); the binding rejects what only the tensors
know."""
import ctypes
import os
import re

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "qr_layer.h")
FAKE = 0x7f0000000000
MB = 1 << 20
NAN, INF = float("nan"), float("inf")


def _qr():
    from quantized_two_stage_amd import qr
    return qr


def test_every_declared_function_is_exported_and_bound():
    qr = _qr()
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(qr_[a-z0-9_]+)\s*\(", src)))
    assert names == ["qr_add_rmsnorm_q8", "qr_gather_add_rmsnorm_q8", "qr_gemm_i8",
                     "qr_gemm_i8_workspace_bytes", "qr_silu_mul_q8"]
    for name in names:
        assert hasattr(qr.LIB, name) and name in qr.EXPORTS and callable(getattr(qr, name))


def _norm(dtype=1, x=FAKE, ldx=64, res=FAKE + MB, ldr=64, w=FAKE + 2 * MB, eps=1e-5, M=4, d=64,
          h=FAKE + 3 * MB, ldh=64, q=FAKE + 4 * MB, ldq=64, s=FAKE + 5 * MB):
    return _qr().LIB.qr_add_rmsnorm_q8(dtype, x, ldx, res, ldr, w, eps, M, d, h, ldh, q, ldq, s,
                                       None)


def _gather(codec=1, dtype=1, wire=FAKE, res=FAKE + MB, ldr=64, w=FAKE + 2 * MB, eps=1e-5, M=4,
            d=64, h=FAKE + 3 * MB, ldh=64, q=FAKE + 4 * MB, ldq=64, s=FAKE + 5 * MB):
    return _qr().LIB.qr_gather_add_rmsnorm_q8(codec, dtype, wire, res, ldr, w, eps, M, d, h, ldh,
                                              q, ldq, s, None)


def _silu(dtype=1, gu=FAKE, ldg=128, M=4, d=64, q=FAKE + MB, ldq=64, s=FAKE + 2 * MB):
    return _qr().LIB.qr_silu_mul_q8(dtype, gu, ldg, M, d, q, ldq, s, None)


def _gemm(dtype=1, a=FAKE, lda=64, sa=FAKE + MB, b=FAKE + 2 * MB, ldb=64, sb=FAKE + 3 * MB,
          bias=None, M=4, N=32, K=64, c=FAKE + 4 * MB, ldc=32, ws=FAKE + 64 * MB, ws_bytes=None):
    qr = _qr()
    need = qr.qr_gemm_i8_workspace_bytes(M, N, K) if ws_bytes is None else ws_bytes
    return qr.LIB.qr_gemm_i8(dtype, a, lda, sa, b, ldb, sb, bias, M, N, K, c, ldc, ws, need, None)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), -2), (dict(dtype=3), -2), (dict(dtype=-1), -2),
    (dict(d=0), -3), (dict(d=131072, ldx=131072, ldr=131072, ldh=131072, ldq=131072), -3),
    (dict(M=(1 << 22) + 1), -3),
    (dict(x=None), -1), (dict(w=None), -1), (dict(q=None), -1), (dict(s=None), -1),
    (dict(res=None), -1), (dict(h=None), -1),               # residual and h come together
    (dict(eps=0.0), -1), (dict(eps=-1.0), -1), (dict(eps=NAN), -1), (dict(eps=INF), -1),
    (dict(ldx=63), -1), (dict(ldr=63), -1), (dict(ldh=0), -1), (dict(ldq=63), -1),
    (dict(ldx=(1 << 40) + 1), -1),
    (dict(x=FAKE + 1), -4), (dict(res=FAKE + MB + 1), -4), (dict(w=FAKE + 2 * MB + 1), -4),
    (dict(h=FAKE + 3 * MB + 1), -4), (dict(s=FAKE + 5 * MB + 2), -4),
    (dict(h=FAKE + 64), -1),                                # h inside x
    (dict(h=FAKE + MB + 2), -1),                            # h over residual, not equal to it
    (dict(h=FAKE + MB, ldh=72), -1),                        # the same start, another stride
    (dict(q=FAKE + 511), -1), (dict(q=FAKE + MB), -1), (dict(q=FAKE + 2 * MB), -1),
    (dict(q=FAKE + 3 * MB), -1), (dict(q=FAKE + 5 * MB), -1),
    (dict(s=FAKE), -1), (dict(s=FAKE + MB + 508), -1), (dict(s=FAKE + 2 * MB), -1),
    (dict(s=FAKE + 3 * MB), -1), (dict(h=FAKE + 2 * MB), -1),
])
def test_norm_rejects(kw, code):
    assert _norm(**kw) == code
    assert _qr().qr_last_error() != ""


@pytest.mark.parametrize("kw,code", [
    (dict(codec=4), -2), (dict(codec=13), -2), (dict(dtype=3), -2),
    (dict(d=60), -3), (dict(d=0), -3), (dict(M=1 << 20, d=1032, ldr=1032, ldh=1032, ldq=1032), -3),
    (dict(wire=None), -1), (dict(wire=FAKE + 8), -4), (dict(h=None), -1), (dict(q=None), -1),
    (dict(res=FAKE + MB + 1), -4), (dict(eps=0.0), -1),
    (dict(h=FAKE + 256), -1),                               # h over the wire's scales
    (dict(q=FAKE + 256), -1), (dict(s=FAKE + 256), -1), (dict(h=FAKE + MB + 16), -1),
])
def test_gather_norm_rejects(kw, code):
    assert _gather(**kw) == code
    assert _qr().qr_last_error() != ""


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), -2), (dict(d=0), -3), (dict(d=131072, ldg=262144, ldq=131072), -3),
    (dict(M=(1 << 22) + 1), -3),
    (dict(gu=None), -1), (dict(q=None), -1), (dict(s=None), -1),
    (dict(ldg=127), -1), (dict(ldq=63), -1), (dict(gu=FAKE + 1), -4), (dict(s=FAKE + MB + 1), -4),
    (dict(q=FAKE + 1000), -1), (dict(s=FAKE), -1), (dict(s=FAKE + MB + 252), -1),
])
def test_silu_rejects(kw, code):
    assert _silu(**kw) == code
    assert _qr().qr_last_error() != ""


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), -2), (dict(K=0), -3), (dict(N=0), -3),
    (dict(K=131072, lda=131072, ldb=131072), -3), (dict(N=(1 << 22) + 1), -3),
    (dict(M=(1 << 22) + 1), -3),
    (dict(a=None), -1), (dict(b=None), -1), (dict(sa=None), -1), (dict(sb=None), -1),
    (dict(c=None), -1), (dict(lda=48), -1), (dict(ldb=48), -1), (dict(ldc=31), -1),
    (dict(lda=72), -4), (dict(ldb=72), -4), (dict(lda=1 << 23), -3), (dict(ldb=1 << 23), -3),
    (dict(a=FAKE + 8), -4), (dict(b=FAKE + 2 * MB + 8), -4), (dict(c=FAKE + 4 * MB + 1), -4),
    (dict(sa=FAKE + MB + 2), -4), (dict(sb=FAKE + 3 * MB + 2), -4),
    (dict(bias=FAKE + 6 * MB + 1), -4), (dict(bias=FAKE + 4 * MB), -1),
    (dict(c=FAKE), -1), (dict(c=FAKE + 2 * MB + 16), -1), (dict(c=FAKE + MB), -1),
    (dict(c=FAKE + 3 * MB), -1),
])
def test_gemm_rejects(kw, code):
    assert _gemm(**kw) == code
    assert _qr().qr_last_error() != ""


def test_a_batch_without_tokens_is_nothing_to_do():
    qr = _qr()
    assert _norm(M=0) == 0 and _norm(M=0, x=None, res=None, h=None, q=None, s=None, w=None) == 0
    assert _gather(M=0) == 0 and _silu(M=0, gu=None) == 0
    assert _gemm(M=0) == 0 and _gemm(M=0, a=None, sa=None, c=None) == 0
    assert qr.qr_last_error() == ""
    assert _norm(M=0, d=0) == -3 and _gemm(M=0, K=0) == -3 and _gather(M=0, d=12) == -3


def test_gemm_workspace_is_checked():
    """wherever a workspace is needed, a missing, short, misaligned or
    overlapping one is rejected"""
    qr = _qr()
    needy = [(M, N, K) for M in (1, 16, 48, 64, 128, 333, 1024) for N in (64, 1000, 2048, 8192)
             for K in (64, 4096, 16384) if qr.qr_gemm_i8_workspace_bytes(M, N, K) > 0]
    for M, N, K in needy:
        need = qr.qr_gemm_i8_workspace_bytes(M, N, K)
        far = dict(M=M, N=N, K=K, lda=K, ldb=K, ldc=N, b=FAKE + (1 << 32), c=FAKE + (1 << 33),
                   sa=FAKE + (1 << 34), sb=FAKE + (1 << 35))
        assert _gemm(ws=FAKE + (1 << 36), ws_bytes=need - 1, **far) == -5
        assert _gemm(ws=None, ws_bytes=need, **far) == -1
        assert _gemm(ws=FAKE + (1 << 36) + 8, ws_bytes=need, **far) == -4
        assert _gemm(ws=FAKE, ws_bytes=need, **far) == -1
        assert _gemm(ws=FAKE + (1 << 33), ws_bytes=need, **far) == -1
    assert qr.qr_gemm_i8_workspace_bytes(0, 64, 64) == 0


def test_binding_rejects_tensors():
    """everything here is refused before a GPU would be needed"""
    qr = _qr()
    f16, i8, f32 = torch.float16, torch.int8, torch.float32
    x, w, s = torch.zeros(2, 16, dtype=f16), torch.zeros(16, dtype=f16), torch.zeros(2)
    q = torch.zeros(2, 16, dtype=i8)
    with pytest.raises(ValueError, match="not on the current GPU"):
        qr.qr_add_rmsnorm_q8(x, x.clone(), w, 1e-5, x.clone(), q, s)
    with pytest.raises(TypeError, match="float16 or bfloat16"):
        qr.qr_add_rmsnorm_q8(x.float(), x, w, 1e-5, x, q, s)
    with pytest.raises(ValueError, match="dimensions"):
        qr.qr_add_rmsnorm_q8(x[0], x, w, 1e-5, x, q, s)
    with pytest.raises(ValueError, match="differ in length"):
        qr.qr_silu_mul_q8(torch.zeros(2, 15, dtype=f16), q, s)
    with pytest.raises(TypeError, match="float16 or bfloat16"):
        qr.qr_gemm_i8(q, s, q, s, torch.zeros(2, 2, dtype=f32))
    with pytest.raises(ValueError, match="not on the current GPU"):
        qr.qr_gemm_i8(q, s, q, s, torch.zeros(2, 2, dtype=f16))
    with pytest.raises(TypeError, match="under dtype"):
        qr.qr_gather_add_rmsnorm_q8(1, q, x, w, 1e-5, x, q, s, dtype=qr.QR_BF16)
    # the checks of single arguments (device -1: tensors in host memory)
    with pytest.raises(ValueError, match="shape"):
        qr._mat("q", q, 2, 15, i8, -1)
    with pytest.raises(TypeError, match="int8"):
        qr._mat("q", x, 2, 16, i8, -1)
    with pytest.raises(ValueError, match="not contiguous"):
        qr._mat("q", q.t(), 16, 2, i8, -1)
    with pytest.raises(ValueError, match="not on GPU"):
        qr._mat("q", q, 2, 16, i8, 0)
    with pytest.raises(ValueError, match="holds 2 values"):
        qr._vec("scales", s, 3, f32, -1)
    with pytest.raises(ValueError, match="not contiguous"):
        qr._vec("scales", torch.zeros(4)[::2], 2, f32, -1)
    # rows of 17 codes: read up to byte 32 of each, which the last row must hold
    wide = torch.zeros(2, 32, dtype=i8)
    assert qr._codes("a", wide[:, :17], 2, 17, -1) == 32
    tight = torch.zeros(32 + 17, dtype=i8).as_strided((2, 17), (32, 1))
    with pytest.raises(ValueError, match="padding"):
        qr._codes("a", tight, 2, 17, -1)
    with pytest.raises(ValueError, match="padding"):
        qr._codes("a", torch.zeros(1, 17, dtype=i8), 1, 17, -1)
    q, s = qr.alloc_q8(3, 17, device="cpu")
    assert q.shape == (3, 17) and q.stride() == (32, 1) and s.shape == (3,)
    assert qr._codes("a", q, 3, 17, -1) == 32
