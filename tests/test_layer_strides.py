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
