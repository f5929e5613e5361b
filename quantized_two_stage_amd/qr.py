"""Python binding of the C ABI in include/qr.h and include/qr_layer.h (argument
marshalling only).

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
           "qr_gemm_i8", "qr_gemm_i8_workspace_bytes")


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
    return _ld(what, t, rows, cols)


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
