"""Row strides that carry no information, and buffers whose rows lie between one another: what the binding and the checks
of arguments accept.  The library's calls below end at a check (a NULL pointer) or launch nothing."""
import pytest
import torch


@pytest.fixture(scope="module")
def qr():
    from quantized_two_stage_amd import qr as q
    return q


def test_the_stride_of_a_single_row_does_not_count(qr):
    """one token's view of a buffer with wide rows: no second row is read, so any stride will do"""
    wide = torch.empty(1 << 23, dtype=torch.int8)
    for ld in (64, 72, 1 << 20, (1 << 23) - 64, 1 << 23, 1 << 45):
        one = wide.as_strided((1, 64), (ld, 1))
        assert qr._codes("a", one, 1, 64, -1) == 64
        assert qr._mat("q", one, 1, 64, torch.int8, -1) == 64
    assert qr._codes("a", wide.as_strided((1, 50), (1 << 23, 1)), 1, 50, -1) == 64
    # two rows: theirs
    assert qr._codes("a", wide.as_strided((2, 64), (80, 1)), 2, 64, -1) == 80
    assert qr._mat("q", wide.as_strided((2, 64), (1 << 20, 1)), 2, 64, torch.int8, -1) == 1 << 20


FAKE, MB = 0x7f0000000000, 1 << 20


def norm_refusal(qr, x=FAKE, ldx=256, h=FAKE + 128, ldh=256, M=4, d=64, q=FAKE + 4 * MB, ldq=64):
    """the text of a refusal of qr_add_rmsnorm_q8: what is looked at last is wrong (h lies over the residual, a value off
    it), so that nothing is launched"""
    assert qr.LIB.qr_add_rmsnorm_q8(1, x, ldx, h + 2, ldh, FAKE + 2 * MB, 1e-5, M, d, h, ldh, q, ldq, FAKE + 5 * MB,
                                    None) == -1
    return qr.qr_last_error()


def test_rows_between_rows_do_not_overlap(qr):
    """columns of one buffer: x and h share its extent but no element"""
    # rows of 128 bytes, 512 apart
    for at in (128, 130, 256, 384, -128, -384, 512 + 128, 2048 - 512 + 128, -512 + 384):
        assert norm_refusal(qr, h=FAKE + at) == "h overlaps residual", at
    for at in (0, 2, 126, 386, 510, -2, -126, 512, 512 + 126, -512, 1536):
        assert norm_refusal(qr, h=FAKE + at) == "h overlaps x", at
    # another stride: rows meet somewhere, or may
    assert norm_refusal(qr, h=FAKE + 128, ldh=264) == "h overlaps x"
    # rows of different types of one stride in bytes: codes between values
    for at in (128, 448, -64, -384):
        assert norm_refusal(qr, q=FAKE + at, ldq=512, h=FAKE + 3 * MB) == "h overlaps residual", at
    for at in (127, 449, -63, 0):
        assert norm_refusal(qr, q=FAKE + at, ldq=512, h=FAKE + 3 * MB) == "q overlaps x", at


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("M,d", [(3, 6), (5, 64), (4, 67), (3, 1000), (3, 1003), (2, 9001), (2, 20004), (2, 33001)])
def test_columns_of_one_buffer(qr, M, d, dtype):
    """x, residual, h, and gate and up, beside one another in rows of one buffer: the bits that buffers of their own give,
    and nothing else written"""
    g = torch.Generator(device="cuda").manual_seed(d)
    buf = torch.randn(M, 5 * d + 7, generator=g, device="cuda").to(dtype)
    w = (1 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(dtype)
    x, res, h, other = (buf[:, 1 + i * d:1 + (i + 1) * d] for i in (0, 1, 2, 3))
    before = buf.clone()
    (q, s), (q2, s2) = qr.alloc_q8(M, d), qr.alloc_q8(M, d)
    h2 = torch.empty(M, d, dtype=dtype, device="cuda")
    qr.qr_add_rmsnorm_q8(x.contiguous(), res.contiguous(), w, 1e-5, h2, q2, s2)
    qr.qr_add_rmsnorm_q8(x, res, w, 1e-5, h, q, s)
    torch.cuda.synchronize()
    assert torch.equal(h, h2) and torch.equal(q, q2) and torch.equal(s, s2)
    keep = torch.ones_like(buf, dtype=torch.bool)
    keep[:, 1 + 2 * d:1 + 3 * d] = False
    assert torch.equal(buf[keep], before[keep])
    # the product writes beside what it does not read
    if d % 16 == 0:
        b, sb = qr.alloc_q8(d, d)
        b.copy_(torch.randint(-127, 128, b.shape, generator=g, device="cuda", dtype=torch.int8))
        sb.fill_(1e-3)
        c = torch.empty(M, d, dtype=dtype, device="cuda")
        qr.qr_gemm_i8(q, s, b, sb, c)
        qr.qr_gemm_i8(q, s, b, sb, other)
        torch.cuda.synchronize()
        assert torch.equal(other, c)
