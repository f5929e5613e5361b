"""Limits of include/qr_f8.h on the host (no GPU needed; the pointers are fake, never touched)."""
import random

import pytest

import f8_tiles
from test_f8_abi import ARG, FAKE, SIZE, _gemm, _norm, _route, _silu, at

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


def _header_allows(E, M, N):
    tiles = -(-M // 256) if E == 0 else M // 256 + min(E, M)
    return tiles * -(-N // 256) < 1 << 23


def test_every_product_that_the_header_allows_fits_a_launch():
    rng = random.Random(1)
    sizes = [(1024, ROWS, 256 * 481, 16), (0, ROWS, 256 * 511, 16), (0, 256, ROWS, 16), (512, 512, ROWS - 65536, 16)]
    while len(sizes) < 20000:
        E = rng.choice([0, 1, 7, 64, 300, 1024])
        M, N = (int(2 ** rng.uniform(0, 22)) for _ in "MN")
        K = int(2 ** rng.uniform(0, 16.99))
        sizes.append((E, M, N, K))
        tiles = -(-M // 256) if E == 0 else M // 256 + min(E, M)
        most = ((1 << 23) - 1) // tiles * 256        # the last N of the limit
        if most <= ROWS:
            sizes.append((E, M, most, K))
    allowed = [s for s in sizes if _header_allows(*s[:3])]
    assert len(allowed) > 15000 and -1 not in f8_tiles.choices(allowed)


def test_more_tiles_than_a_launch_holds():
    far = dict(a=1 << 46, sa=1 << 47, b=1 << 48, sb=1 << 50, c=1 << 52)
    M, N = ROWS, 512 * 256
    assert not _header_allows(0, M, N)
    assert _gemm(M=M, N=N, K=16, lda=16, ldb=16, ldsa=4, ldc=N, **far) == SIZE
