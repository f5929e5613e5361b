"""Limits of include/qr_f8.h on the host (no GPU needed; the pointers are fake, never touched)."""
import pytest

from test_f8_abi import ARG, FAKE, _norm, _route, _silu, at

ROWS, STRIDE = 1 << 22, 1 << 40                      # the most that there may be


@pytest.mark.parametrize("call,kw", [
    # binary32 rows whose extent is nearly 2^64 bytes, and another buffer inside it
    (_silu, dict(M=ROWS, s=FAKE, lds=STRIDE, gu=at(1), q=FAKE - (1 << 40))),
    (_silu, dict(M=ROWS, s=FAKE, lds=STRIDE, gu=FAKE - (1 << 45), q=at(1))),
    (_norm, dict(M=ROWS, x=at(1 << 24), res=None, h=None, y=None, w=at(1 << 26), q=FAKE - (1 << 40), s=FAKE, lds=STRIDE)),
    (_route, dict(dtype=3, T=ROWS, k=1, x=FAKE, ldl=STRIDE, w=at(100), e=at(200), o=at(300), r=at(400), p=at(500),
                  ws=at(600))),
])
def test_extents_near_the_end_of_the_address_space(call, kw):
    assert call(**kw) == ARG
