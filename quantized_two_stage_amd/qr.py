"""Python binding of the C ABI in include/qr.h, include/qr_layer.h and
include/qr_f8.h (argument marshalling only).

Every function has the name of the C entry point it calls and takes torch
tensors on the GPU; all work happens in libqr.so's HIP kernels, on the current
torch stream unless `stream` is given.  There is no other implementation: if
libqr.so is missing this module raises on import.  Since the C ABI sees only
pointers, each function first checks what only the tensors know (enough
bytes behind every pointer, contiguous, in device memory, as many outputs as
inputs) and raises ValueError before any call.
"""
import ctypes
import os

import torch

QR_FP, QR_Q8, QR_Q6, QR_Q4, QR_FP8 = 0, 1, 2, 3, 5
QR_Q8_ASYM, QR_Q6_ASYM, QR_Q4_ASYM = 9, 10, 11
QR_FP16, QR_BF16, QR_BF16_VIA_FP16 = 0, 1, 2
QR_FP32 = 3                                # of a router's logits only
CODECS = (QR_FP, QR_FP8, QR_Q8, QR_Q6, QR_Q4, QR_Q8_ASYM, QR_Q6_ASYM, QR_Q4_ASYM)
CODEC_NAMES = {QR_FP: "fp", QR_Q8: "q8", QR_Q6: "q6", QR_Q4: "q4", QR_FP8: "fp8",
               QR_Q8_ASYM: "q8a", QR_Q6_ASYM: "q6a", QR_Q4_ASYM: "q4a"}
ERRORS = {-1: "QR_ERR_ARG", -2: "QR_ERR_UNSUPPORTED", -3: "QR_ERR_SIZE",
          -4: "QR_ERR_ALIGN", -5: "QR_ERR_WORKSPACE", -6: "QR_ERR_HIP"}
QR_MAX_BYTES = 1 << 31
QR_SCRATCH_BYTES = 64 << 20

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libqr.so")


class QRError(RuntimeError):
    def __init__(self, code, msg):
        super().__init__("%s (%d): %s" % (ERRORS.get(code, "?"), code, msg))
        self.code = code


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError("libqr.so is not built (%s); run "
                          "quantized_two_stage_amd/build.py" % LIB_PATH)
    L = ctypes.CDLL(LIB_PATH)
    sz, i32, f32, P = ctypes.c_size_t, ctypes.c_int, ctypes.c_float, ctypes.c_void_p
    PP = ctypes.POINTER(ctypes.c_void_p)
    sig = {
        "qr_wire_bytes": (sz, [i32, sz]),
        "qr_sim_workspace_bytes": (sz, [i32, i32, sz]),
        "qr_recv_bytes": (sz, [i32, i32, sz]),
        "qr_quantize_recv": (i32, [i32, i32, i32, PP, sz, P, P]),
        "qr_reduce_recv": (i32, [i32, i32, i32, P, sz, i32, P, P]),
        "qr_quantize": (i32, [i32, i32, P, sz, P, P]),
        "qr_dequantize": (i32, [i32, i32, P, sz, P, P]),
        "qr_quantize_ranks": (i32, [i32, i32, i32, PP, sz, PP, P]),
        "qr_reduce_stage1": (i32, [i32, i32, i32, PP, sz, i32, P, P]),
        "qr_gather_stage2": (i32, [i32, i32, i32, P, sz, PP, P]),
        "qr_allreduce_sim": (i32, [i32, i32, i32, PP, PP, sz, P, sz, P]),
        "qr_allreduce_oneshot": (i32, [i32, i32, PP, PP, sz, P]),
        "qr_allreduce_sim_noalloc": (i32, [i32, i32, i32, PP, PP, sz, P]),
        "qr_last_error": (ctypes.c_char_p, []),
        "qr_add_rmsnorm_q8": (i32, [i32, P, sz, P, sz, P, f32, sz, sz, P, sz, P, sz, P, P]),
        "qr_gather_add_rmsnorm_q8": (i32, [i32, i32, P, P, sz, P, f32, sz, sz, P, sz, P, sz, P,
                                           P]),
        "qr_silu_mul_q8": (i32, [i32, P, sz, sz, sz, P, sz, P, P]),
        "qr_gemm_i8": (i32, [i32, P, sz, P, P, sz, P, P, sz, sz, sz, P, sz, P, sz, P]),
        "qr_gemm_i8_workspace_bytes": (sz, [sz, sz, sz]),
        "qr_add_rmsnorm_f8": (i32, [i32, P, sz, P, sz, P, f32, sz, sz, P, sz, P, sz, P, sz, P, sz,
                                    P]),
        "qr_silu_mul_f8": (i32, [i32, P, sz, sz, sz, P, sz, P, sz, P]),
        "qr_gemm_f8": (i32, [i32, P, sz, P, sz, P, sz, P, sz, P, sz, sz, sz, P, sz, P]),
        "qr_gemm_f8_grouped": (i32, [i32, P, sz, P, sz, P, sz, P, sz, sz, P, sz, sz, P, sz, P, sz,
                                     sz, sz, sz, P, sz, P]),
        "qr_route": (i32, [i32, P, sz, sz, sz, sz, i32, P, P, P, P, P, P, sz, P]),
        "qr_route_workspace_bytes": (sz, [sz, sz, sz]),
        "qr_combine": (i32, [i32, P, sz, sz, P, P, sz, sz, sz, P, sz, P, sz, P]),
    }
    for name, (res, args) in sig.items():
        f = getattr(L, name)
        f.restype, f.argtypes = res, args
    return L


LIB = _load()
EXPORTS = ("qr_wire_bytes", "qr_sim_workspace_bytes", "qr_recv_bytes", "qr_quantize",
           "qr_dequantize", "qr_quantize_ranks", "qr_quantize_recv", "qr_reduce_stage1",
           "qr_reduce_recv", "qr_gather_stage2",
           "qr_allreduce_sim", "qr_allreduce_oneshot", "qr_allreduce_sim_noalloc",
           "qr_last_error", "qr_add_rmsnorm_q8", "qr_gather_add_rmsnorm_q8", "qr_silu_mul_q8",
           "qr_gemm_i8", "qr_gemm_i8_workspace_bytes", "qr_add_rmsnorm_f8", "qr_silu_mul_f8",
           "qr_gemm_f8", "qr_gemm_f8_grouped", "qr_route", "qr_route_workspace_bytes",
           "qr_combine")


def _check(rc):
    if rc != 0:
        raise QRError(rc, LIB.qr_last_error().decode())


def _dtype_of(t, dtype):
    if dtype is not None:
        return dtype
    if t.dtype == torch.float16:
        return QR_FP16
    if t.dtype == torch.bfloat16:
        return QR_BF16
    raise TypeError("pass dtype= for a %s buffer" % t.dtype)


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else stream)


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else ctypes.c_void_p(0)


def _ptrs(ts):
    return (ctypes.c_void_p * len(ts))(*[t.data_ptr() for t in ts])


def _n16(t):
    return t.numel() * t.element_size() // 2


def _nbytes(t):
    return t.numel() * t.element_size()


def _bufs(*groups):
    """The C ABI sees only pointers: refuse, before any call, a tensor the
    kernels would run past (too small or not contiguous) or one not in
    device memory.  groups: (name, tensors, bytes each must hold)."""
    for what, ts, need in groups:
        for i, t in enumerate(ts):
            if not t.is_contiguous():
                raise ValueError("%s[%d] is not contiguous" % (what, i))
            if _nbytes(t) < need:
                raise ValueError("%s[%d] holds %d bytes, %d needed" % (what, i, _nbytes(t),
                                                                       need))
    for what, ts, _ in groups:
        for i, t in enumerate(ts):
            if not t.is_cuda:
                raise ValueError("%s[%d] is not in GPU memory" % (what, i))


def _same_count(xs, ys, a, b):
    if len(xs) != len(ys):
        raise ValueError("%d %s but %d %s" % (len(xs), a, len(ys), b))


def qr_last_error():
    return LIB.qr_last_error().decode()


def qr_wire_bytes(codec, n):
    return LIB.qr_wire_bytes(codec, n)


def qr_sim_workspace_bytes(W, codec, n):
    return LIB.qr_sim_workspace_bytes(W, codec, n)


def qr_recv_bytes(W, codec, n):
    return LIB.qr_recv_bytes(W, codec, n)


def qr_quantize(codec, x, wire, dtype=None, stream=None):
    n = _n16(x)
    _bufs(("x", [x], 2 * n), ("wire", [wire], qr_wire_bytes(codec, n)))
    _check(LIB.qr_quantize(codec, _dtype_of(x, dtype), _ptr(x), _n16(x), _ptr(wire),
                           _stream(stream)))
    return wire


def qr_dequantize(codec, wire, y, dtype=None, stream=None):
    n = _n16(y)
    _bufs(("wire", [wire], qr_wire_bytes(codec, n)), ("y", [y], 2 * n))
    _check(LIB.qr_dequantize(codec, _dtype_of(y, dtype), _ptr(wire), _n16(y), _ptr(y),
                             _stream(stream)))
    return y


def qr_quantize_ranks(codec, xs, wires, dtype=None, stream=None):
    _same_count(xs, wires, "inputs", "wire images")
    n = _n16(xs[0])
    _bufs(("xs", xs, 2 * n), ("wires", wires, qr_wire_bytes(codec, n)))
    _check(LIB.qr_quantize_ranks(codec, _dtype_of(xs[0], dtype), len(xs), _ptrs(xs),
                                 _n16(xs[0]), _ptrs(wires), _stream(stream)))
    return wires


def qr_quantize_recv(codec, xs, recv, dtype=None, stream=None):
    """stage 0 of W ranks into one receive buffer (qr_recv_bytes bytes)"""
    n = _n16(xs[0])
    _bufs(("xs", xs, 2 * n), ("recv", [recv], qr_recv_bytes(len(xs), codec, n)))
    _check(LIB.qr_quantize_recv(codec, _dtype_of(xs[0], dtype), len(xs), _ptrs(xs), n,
                                _ptr(recv), _stream(stream)))
    return recv


def qr_reduce_recv(codec, W, recv, n, reduced, dtype, owner=-1, stream=None):
    """stage 1 of W ranks from a receive buffer"""
    _bufs(("recv", [recv], qr_recv_bytes(W, codec, n)),
          ("reduced", [reduced], qr_wire_bytes(codec, n)))
    _check(LIB.qr_reduce_recv(codec, dtype, W, _ptr(recv), n, owner, _ptr(reduced),
                              _stream(stream)))
    return reduced


def qr_reduce_stage1(codec, wires, n, reduced, dtype, owner=-1, stream=None):
    _bufs(("wires", wires, qr_wire_bytes(codec, n)),
          ("reduced", [reduced], qr_wire_bytes(codec, n)))
    _check(LIB.qr_reduce_stage1(codec, dtype, len(wires), _ptrs(wires), n, owner,
                                _ptr(reduced), _stream(stream)))
    return reduced


def qr_gather_stage2(codec, reduced, ys, dtype=None, stream=None):
    n = _n16(ys[0])
    _bufs(("reduced", [reduced], qr_wire_bytes(codec, n)), ("ys", ys, 2 * n))
    _check(LIB.qr_gather_stage2(codec, _dtype_of(ys[0], dtype), len(ys), _ptr(reduced),
                                _n16(ys[0]), _ptrs(ys), _stream(stream)))
    return ys


def qr_allreduce_sim(codec, xs, ys, workspace, dtype=None, stream=None):
    """ys[r] = the simulated two-stage allreduce of xs (out-of-place)."""
    _same_count(xs, ys, "inputs", "outputs")
    n = _n16(xs[0])
    # the workspace's size is passed to the call, which checks it
    _bufs(("xs", xs, 2 * n), ("ys", ys, 2 * n), ("workspace", [workspace], 0))
    ws_bytes = _nbytes(workspace)
    _check(LIB.qr_allreduce_sim(len(xs), _dtype_of(xs[0], dtype), codec, _ptrs(xs),
                                _ptrs(ys), n, _ptr(workspace), ws_bytes, _stream(stream)))
    return ys


def qr_allreduce_sim_noalloc(codec, xs, ys, dtype=None, stream=None):
    """qr_allreduce_sim with the library's own workspace buffer: allocates
    nothing (for callers that cannot); calls on one GPU must not overlap."""
    _same_count(xs, ys, "inputs", "outputs")
    n = _n16(xs[0])
    _bufs(("xs", xs, 2 * n), ("ys", ys, 2 * n))
    _check(LIB.qr_allreduce_sim_noalloc(len(xs), _dtype_of(xs[0], dtype), codec, _ptrs(xs),
                                        _ptrs(ys), n, _stream(stream)))
    return ys


def qr_allreduce_oneshot(xs, ys, dtype=None, stream=None):
    """ys[r] = the one-stage allreduce of xs: every rank sums all W buffers."""
    _same_count(xs, ys, "inputs", "outputs")
    n = _n16(xs[0])
    _bufs(("xs", xs, 2 * n), ("ys", ys, 2 * n))
    _check(LIB.qr_allreduce_oneshot(len(xs), _dtype_of(xs[0], dtype), _ptrs(xs), _ptrs(ys),
                                    _n16(xs[0]), _stream(stream)))
    return ys


def alloc_wire(codec, n, device="cuda"):
    """A device buffer for one wire image (padding bytes start at zero)."""
    return torch.zeros(qr_wire_bytes(codec, n), dtype=torch.uint8, device=device)


def alloc_recv(W, codec, n, device="cuda"):
    """A device buffer for a receive buffer (padding bytes start at zero)."""
    return torch.zeros(qr_recv_bytes(W, codec, n), dtype=torch.uint8, device=device)


def alloc_workspace(W, codec, n, device="cuda"):
    return torch.empty(qr_sim_workspace_bytes(W, codec, n), dtype=torch.uint8,
                       device=device)


# ---------------------------------------------------------------------------
# the operators between two allreduces (include/qr_layer.h)

_DTYPES = {torch.float16: QR_FP16, torch.bfloat16: QR_BF16}


def _type16(t, what):
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise TypeError("%s is %s: float16 or bfloat16 expected" % (what, t.dtype))
    return code


def _refuse(what, t, dtype, dev, shape):
    if t.dtype is not dtype:
        raise TypeError("%s is %s: %s expected" % (what, t.dtype, dtype))
    if t.get_device() != dev:
        raise ValueError("%s is not on GPU %d" % (what, dev))
    raise ValueError(shape)


def _mat(what, t, rows, cols, dtype, dev):
    """A matrix argument: its row stride in elements (rows contiguous)."""
    if t.dtype is not dtype or t.get_device() != dev or t.shape != (rows, cols):
        _refuse(what, t, dtype, dev,
                "%s has shape %s: %s expected" % (what, tuple(t.shape), (rows, cols)))
    ld, step = t.stride()
    if step != 1 and cols > 1:
        raise ValueError("%s: the values of a row are not contiguous" % what)
    return ld if rows > 1 else cols


def _ld(what, t, rows, cols):
    """The row stride of a matrix whose shape, type and device are known (of a
    single row the shortest there is: its own says nothing)."""
    ld, step = t.stride()
    if step != 1 and cols > 1:
        raise ValueError("%s: the values of a row are not contiguous" % what)
    return ld if rows > 1 else cols


def _vec(what, t, n, dtype, dev):
    if t.dtype is not dtype or t.get_device() != dev or t.numel() != n:
        _refuse(what, t, dtype, dev, "%s holds %d values: %d expected" % (what, t.numel(), n))
    if not t.is_contiguous():
        raise ValueError("%s is not contiguous" % what)
    return t.data_ptr()


def _codes(what, t, rows, cols, dev):
    """A matrix of codes that qr_gemm_i8 reads: rows of whole 16-byte pieces,
    the last one's padding inside the tensor's storage."""
    ld = _mat(what, t, rows, cols, torch.int8, dev)
    if rows == 1:
        ld = -(-cols // 16) * 16
    if cols % 16 and rows > 0 and (t.storage_offset() + (rows - 1) * ld + -(-cols // 16) * 16
                                   > t.untyped_storage().nbytes()):
        raise ValueError("%s: the padding of its last row up to a multiple of 16 is outside "
                         "its storage (alloc_q8 makes room for it)" % what)
    return ld


def _device(t, what):
    """The current GPU, which the tensors of a call must be on."""
    dev = t.get_device()
    if dev < 0 or dev != torch._C._cuda_getDevice():
        raise ValueError("%s is not on the current GPU" % what)
    return dev


def _stream_on(dev, stream):
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else stream


def _matrix_shape(what, t):
    if t.dim() != 2:
        raise ValueError("%s has %d dimensions: a matrix expected" % (what, t.dim()))
    return t.shape


def _norm_args(residual, weight, h, q, scales, M, d, dtype, dev):
    ldr = _mat("residual", residual, M, d, dtype, dev) if residual is not None else 0
    ldh = _mat("h", h, M, d, dtype, dev) if h is not None else 0
    return (residual.data_ptr() if residual is not None else None, ldr,
            _vec("weight", weight, d, dtype, dev),
            h.data_ptr() if h is not None else None, ldh,
            q.data_ptr(), _mat("q", q, M, d, torch.int8, dev),
            _vec("scales", scales, M, torch.float32, dev))


def qr_add_rmsnorm_q8(x, residual, weight, eps, h, q, scales, stream=None):
    """h = x + residual; q, scales = the 8-bit codes and row scales of h's
    root-mean-square norm times weight.  residual and h may be one tensor
    (updated in place), or both None (h = x).  Matrices are [M, d] with
    contiguous rows, scales holds M float32."""
    M, d = _matrix_shape("x", x)
    code = _type16(x, "x")
    dev = _device(x, "x")
    ldx = _ld("x", x, M, d)
    pr, ldr, pw, ph, ldh, pq, ldq, ps = _norm_args(residual, weight, h, q, scales, M, d, x.dtype,
                                                   dev)
    _check(LIB.qr_add_rmsnorm_q8(code, x.data_ptr(), ldx, pr, ldr, pw, eps, M, d, ph, ldh, pq,
                                 ldq, ps, _stream_on(dev, stream)))
    return h, q, scales


def qr_gather_add_rmsnorm_q8(codec, wire, residual, weight, eps, h, q, scales, dtype=None,
                             stream=None):
    """qr_add_rmsnorm_q8 of the values that a wire image of h.numel() elements
    holds (residual may be None: h = the values).  dtype: QR_BF16_VIA_FP16 for
    bfloat16 buffers under the cast option."""
    M, d = _matrix_shape("h", h)
    code = _type16(h, "h") if dtype is None else dtype
    if h.dtype is not (torch.float16 if code == QR_FP16 else torch.bfloat16):
        raise TypeError("h is %s under dtype %d" % (h.dtype, code))
    dev = _device(h, "h")
    if wire.get_device() != dev or not wire.is_contiguous():
        raise ValueError("wire is not contiguous on GPU %d" % dev)
    if M * d > 0 and _nbytes(wire) < qr_wire_bytes(codec, M * d):
        raise ValueError("wire holds %d bytes, %d needed" % (_nbytes(wire),
                                                             qr_wire_bytes(codec, M * d)))
    pr, ldr, pw, ph, ldh, pq, ldq, ps = _norm_args(residual, weight, h, q, scales, M, d, h.dtype,
                                                   dev)
    _check(LIB.qr_gather_add_rmsnorm_q8(codec, code, wire.data_ptr(), pr, ldr, pw, eps, M, d, ph,
                                        ldh, pq, ldq, ps, _stream_on(dev, stream)))
    return h, q, scales


def qr_silu_mul_q8(gu, q, scales, stream=None):
    """q, scales = the 8-bit codes and row scales of silu(gate) * up, where a
    row of gu ([M, 2d]) holds the d gate values and then the d up values."""
    M, d2 = _matrix_shape("gu", gu)
    if d2 % 2 != 0:
        raise ValueError("gu has rows of %d values: gate and up differ in length" % d2)
    d = d2 // 2
    code = _type16(gu, "gu")
    dev = _device(gu, "gu")
    _check(LIB.qr_silu_mul_q8(code, gu.data_ptr(), _ld("gu", gu, M, d2), M, d,
                              q.data_ptr(), _mat("q", q, M, d, torch.int8, dev),
                              _vec("scales", scales, M, torch.float32, dev),
                              _stream_on(dev, stream)))
    return q, scales


def qr_gemm_i8(a, sa, b, sb, c, bias=None, workspace=None, stream=None):
    """c = (a @ b^T in 32-bit integers) * sa * sb (+ bias), rounded once to c's
    type.  a: [M, K] int8 codes of the tokens and sa their M float32 scales,
    b: [N, K] int8 codes of the weights and sb their N scales.  No size needs a
    workspace; one that is passed is left alone."""
    M, K = _matrix_shape("a", a)
    N = _matrix_shape("b", b)[0]
    code = _type16(c, "c")
    dev = _device(c, "c")
    _check(LIB.qr_gemm_i8(
        code, a.data_ptr(), _codes("a", a, M, K, dev), _vec("sa", sa, M, torch.float32, dev),
        b.data_ptr(), _codes("b", b, N, K, dev), _vec("sb", sb, N, torch.float32, dev),
        _vec("bias", bias, N, c.dtype, dev) if bias is not None else None, M, N, K,
        c.data_ptr(), _mat("c", c, M, N, c.dtype, dev),
        workspace.data_ptr() if workspace is not None else None,
        _workspace_bytes(workspace, dev), _stream_on(dev, stream)))
    return c


def _workspace_bytes(t, dev):
    if t is None:
        return 0
    if t.get_device() != dev or not t.is_contiguous():
        raise ValueError("workspace is not contiguous on GPU %d" % dev)
    return _nbytes(t)


def qr_gemm_i8_workspace_bytes(M, N, K):
    return LIB.qr_gemm_i8_workspace_bytes(M, N, K)


def alloc_gemm_workspace(M, N, K, device="cuda"):
    """Device memory for qr_gemm_i8's workspace (None where it needs none)."""
    n = qr_gemm_i8_workspace_bytes(M, N, K)
    return torch.empty(n, dtype=torch.uint8, device=device) if n else None


def alloc_q8(M, d, device="cuda"):
    """Device buffers for M rows of d codes, each row starting at a multiple of
    16 bytes as qr_gemm_i8 reads them, and for the M scales."""
    q = torch.empty(M, -(-d // 16) * 16, dtype=torch.int8, device=device)[:, :d]
    return q, torch.empty(M, dtype=torch.float32, device=device)


# ---------------------------------------------------------------------------
# the operators in 8-bit floating point, dense and by experts (include/qr_f8.h)

_F8 = torch.float8_e4m3fn
_LOGITS = {torch.float16: QR_FP16, torch.bfloat16: QR_BF16, torch.float32: QR_FP32}


def _blocks(n):
    return -(-n // 128)


def _pieces(what, t, rows, cols, dtype, dev, piece):
    """A matrix whose rows are read in whole pieces of `piece` elements (16
    bytes), the last one's padding inside the tensor's storage."""
    ld = _mat(what, t, rows, cols, dtype, dev)
    padded = -(-cols // piece) * piece
    if rows == 1:
        ld = padded
    if cols % piece and rows > 0 and ((t.storage_offset() + (rows - 1) * ld + padded)
                                      * t.element_size() > t.untyped_storage().nbytes()):
        raise ValueError("%s: the padding of its last row up to a multiple of %d is outside its "
                         "storage (alloc_f8 makes room for it)" % (what, piece))
    return ld


def _table(what, t, rows, cols, dtype, dev):
    """A contiguous matrix argument."""
    if t.dtype is not dtype or t.get_device() != dev or t.shape != (rows, cols):
        _refuse(what, t, dtype, dev,
                "%s has shape %s: %s expected" % (what, tuple(t.shape), (rows, cols)))
    if not t.is_contiguous():
        raise ValueError("%s is not contiguous" % what)
    return t.data_ptr()


def qr_add_rmsnorm_f8(x, residual, weight, eps, h, y, q, scales, stream=None):
    """h = x + residual; q, scales = the e4m3 codes and block scales of h's
    root-mean-square norm times weight; y (or None) these values in 16 bits.
    residual and h may be one tensor (updated in place), or both None (h = x).
    Matrices are [M, d] with contiguous rows, scales [M, ceil(d/128)] float32."""
    M, d = _matrix_shape("x", x)
    code = _type16(x, "x")
    dev = _device(x, "x")
    ldx = _ld("x", x, M, d)
    ldr = _mat("residual", residual, M, d, x.dtype, dev) if residual is not None else 0
    ldh = _mat("h", h, M, d, x.dtype, dev) if h is not None else 0
    ldy = _mat("y", y, M, d, x.dtype, dev) if y is not None else 0
    _check(LIB.qr_add_rmsnorm_f8(
        code, x.data_ptr(), ldx, residual.data_ptr() if residual is not None else None, ldr,
        _vec("weight", weight, d, x.dtype, dev), eps, M, d,
        h.data_ptr() if h is not None else None, ldh, y.data_ptr() if y is not None else None, ldy,
        q.data_ptr(), _mat("q", q, M, d, _F8, dev), scales.data_ptr(),
        _mat("scales", scales, M, _blocks(d), torch.float32, dev), _stream_on(dev, stream)))
    return h, y, q, scales


def qr_silu_mul_f8(gu, q, scales, stream=None):
    """q, scales = the e4m3 codes and block scales of silu(gate) * up, where a
    row of gu ([M, 2d]) holds the d gate values and then the d up values."""
    M, d2 = _matrix_shape("gu", gu)
    if d2 % 2 != 0:
        raise ValueError("gu has rows of %d values: gate and up differ in length" % d2)
    d = d2 // 2
    code = _type16(gu, "gu")
    dev = _device(gu, "gu")
    _check(LIB.qr_silu_mul_f8(code, gu.data_ptr(), _ld("gu", gu, M, d2), M, d, q.data_ptr(),
                              _mat("q", q, M, d, _F8, dev), scales.data_ptr(),
                              _mat("scales", scales, M, _blocks(d), torch.float32, dev),
                              _stream_on(dev, stream)))
    return q, scales


def qr_gemm_f8(a, sa, b, sb, c, bias=None, stream=None):
    """c = a @ b^T (+ bias) of e4m3 codes, rounded once to c's type.  a: [M, K]
    and sa its [M, ceil(K/128)] float32 block scales, b: [N, K] and sb its
    [ceil(N/128), ceil(K/128)] scales of blocks of 128 x 128."""
    M, K = _matrix_shape("a", a)
    N = _matrix_shape("b", b)[0]
    code = _type16(c, "c")
    dev = _device(c, "c")
    kb = _blocks(K)
    _check(LIB.qr_gemm_f8(
        code, a.data_ptr(), _pieces("a", a, M, K, _F8, dev, 16), sa.data_ptr(),
        _pieces("sa", sa, M, kb, torch.float32, dev, 4), b.data_ptr(),
        _pieces("b", b, N, K, _F8, dev, 16), sb.data_ptr(),
        _mat("sb", sb, _blocks(N), kb, torch.float32, dev),
        _vec("bias", bias, N, c.dtype, dev) if bias is not None else None, M, N, K, c.data_ptr(),
        _mat("c", c, M, N, c.dtype, dev), _stream_on(dev, stream)))
    return c


def qr_gemm_f8_grouped(a, sa, b, sb, offsets, c, rows=None, bias=None, stream=None):
    """The products of E experts: rows offsets[e] to offsets[e + 1] of c ([M, N])
    are those of a, or with `rows` ([M] int32) row i is a's row rows[i], times
    b[e]^T (+ bias[e]).  b: [E, N, K] e4m3 codes, sb: [E, ceil(N/128),
    ceil(K/128)], bias: [E, N], offsets: [E + 1] int32 on the GPU."""
    tokens, K = _matrix_shape("a", a)
    M, N = _matrix_shape("c", c)
    code = _type16(c, "c")
    dev = _device(c, "c")
    kb = _blocks(K)
    for what, t in (("b", b), ("sb", sb)):
        if t.dim() != 3:
            raise ValueError("%s has %d dimensions: one matrix for each expert expected"
                             % (what, t.dim()))
    E = b.shape[0]
    if sb.shape[0] != E:
        raise ValueError("sb holds %d experts' scales: %d expected" % (sb.shape[0], E))
    if E == 0:
        raise ValueError("b holds no expert")
    if rows is None and tokens != M:
        raise ValueError("a has %d rows, c %d" % (tokens, M))
    # the padding that may be missing is that of the last expert's last row
    ldb = _pieces("b", b[-1], N, K, _F8, dev, 16)
    ldsb = _mat("sb", sb[0], _blocks(N), kb, torch.float32, dev)
    ldbias = _mat("bias", bias, E, N, c.dtype, dev) if bias is not None else 0
    _check(LIB.qr_gemm_f8_grouped(
        code, a.data_ptr(), _pieces("a", a, tokens, K, _F8, dev, 16), sa.data_ptr(),
        _pieces("sa", sa, tokens, kb, torch.float32, dev, 4),
        _vec("rows", rows, M, torch.int32, dev) if rows is not None else None, tokens,
        b.data_ptr(), ldb, b.stride(0) if E > 1 else 0, sb.data_ptr(), ldsb,
        sb.stride(0) if E > 1 else 0, bias.data_ptr() if bias is not None else None, ldbias,
        _vec("offsets", offsets, E + 1, torch.int32, dev), E, M, N, K, c.data_ptr(),
        _mat("c", c, M, N, c.dtype, dev), _stream_on(dev, stream)))
    return c


def qr_route(logits, weights, experts, offsets, rows, place, renormalize=False, workspace=None,
             stream=None):
    """The k experts of the largest logits ([T, E]) of every token, in falling
    order: experts [T, k] int32 and their softmax weights [T, k] float32 (over all
    experts, or with renormalize over the k); the rows sorted by expert: offsets
    [E + 1], rows [T * k] (each row's token) and place [T, k] (each choice's row),
    int32.  workspace: alloc_route_workspace(T, E, k)."""
    T, E = _matrix_shape("logits", logits)
    code = _LOGITS.get(logits.dtype)
    if code is None:
        raise TypeError("logits are %s: float16, bfloat16 or float32 expected" % logits.dtype)
    dev = _device(logits, "logits")
    k = _matrix_shape("weights", weights)[1]
    _check(LIB.qr_route(
        code, logits.data_ptr(), _ld("logits", logits, T, E), T, E, k, int(bool(renormalize)),
        _table("weights", weights, T, k, torch.float32, dev),
        _table("experts", experts, T, k, torch.int32, dev),
        _vec("offsets", offsets, E + 1, torch.int32, dev),
        _vec("rows", rows, T * k, torch.int32, dev), _table("place", place, T, k, torch.int32, dev),
        workspace.data_ptr() if workspace is not None else None, _workspace_bytes(workspace, dev),
        _stream_on(dev, stream)))
    return weights, experts, offsets, rows, place


def qr_combine(c, place, weights, y, addend=None, stream=None):
    """y[t] = sum_j weights[t][j] * c[place[t][j]] (+ addend[t]).  c: [R, d],
    place [T, k] int32 (places outside c add nothing), weights [T, k] float32,
    y and addend [T, d]; addend may be y itself."""
    R, d = _matrix_shape("c", c)
    code = _type16(c, "c")
    dev = _device(y, "y")
    T, k = _matrix_shape("place", place)
    lda = _mat("addend", addend, T, d, c.dtype, dev) if addend is not None else 0
    _check(LIB.qr_combine(
        code, c.data_ptr(), _mat("c", c, R, d, c.dtype, dev), R,
        _vec("place", place, T * k, torch.int32, dev),
        _table("weights", weights, T, k, torch.float32, dev), T, k, d,
        addend.data_ptr() if addend is not None else None, lda, y.data_ptr(),
        _mat("y", y, T, d, c.dtype, dev), _stream_on(dev, stream)))
    return y


def qr_route_workspace_bytes(T, E, k):
    return LIB.qr_route_workspace_bytes(T, E, k)


def alloc_route_workspace(T, E, k, device="cuda"):
    """Device memory for qr_route's workspace (None where it needs none)."""
    n = qr_route_workspace_bytes(T, E, k)
    return torch.empty(n, dtype=torch.uint8, device=device) if n else None


def alloc_f8(M, d, device="cuda"):
    """Device buffers for M rows of d e4m3 codes and for their block scales, each
    row starting at a multiple of 16 bytes as qr_gemm_f8 reads them."""
    q = torch.empty(M, -(-d // 16) * 16, dtype=_F8, device=device)[:, :d]
    return q, torch.empty(M, -(-_blocks(d) // 4) * 4, dtype=torch.float32, device=device)[:, :_blocks(d)]
