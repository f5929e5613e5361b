"""Which kernels of include/qr_f8.h the library holds: those that a call can reach, and no others (no GPU needed)."""
import re

import f8_tiles
from f8_edges import ROUTES, kernel_of_route

from quantized_two_stage_amd import qr

TYPES = (0, 1)                                       # of 16 bits
EXPERTS = (1, 8, 64, 65, 128, 129, 256, 257, 512, 513, 1024)
TOKENS = (1, 16, 17, 32, 33, 64, 65, 5000)


def held(kernel, *kinds):
    """the template arguments of a kernel's instances in the library, from their mangled names"""
    args = "".join("L%s(-?[n0-9]+)E" % kind for kind in kinds)
    found = re.findall((kernel + "I" + args + "E").encode(), open(qr.LIB_PATH, "rb").read())
    return {tuple(int(x) for x in f) for f in found}


def test_router():
    reached = set()
    for dtype in (*TYPES, 3):
        for E in EXPERTS:
            for T in TOKENS:
                reached.add((dtype, *kernel_of_route(T, E)))
    assert held("k_choose", *"iiiib") == reached
    assert {x[1:] for x in reached} == {kernel_of_route(T, E) for T, E, _ in ROUTES}       # each has a test


def test_products():
    split, tile = held("k_split_f8", *"iiiiibb"), held("k_tile_f8", *"iiiiiibb")
    assert {x[:2] for x in split | tile} == {t[:2] for t in f8_tiles.tiles()}
    # one product takes tiles of 8 rows up to 8 tokens only, whose weights are read by one workgroup alone
    assert {x[5:] for x in split if x[0] == 8} == {(1, 0), (1, 1), (0, 1)}
    for kernels in (split, tile):
        for x in kernels:
            if x[0] != 8:
                assert {x[:-2] + (once, grouped) for once in (0, 1) for grouped in (0, 1)} <= kernels
