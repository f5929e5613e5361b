"""Which kernels of include/qr_f8.h the library holds: those that a call can reach, and no others (no GPU needed)."""
import re

import f8_tiles

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
                # lanes to a token and logits to a lane
                G, V = ((8, 8) if E <= 64 else (16, 8) if E <= 128 else (16, 16) if E <= 256 else (64, 16) if E > 512 else
                        (64, 8) if T <= 16 else (16, 32))
                lanes = 256 if T <= 64 and E <= 256 and T * G <= 256 else 1024
                reached.add((dtype, G, V, lanes, int(T <= 64)))
    assert held("k_choose", *"iiiib") == reached


def test_products():
    split, tile = held("k_split_f8", *"iiiiibb"), held("k_tile_f8", *"iiiiiibb")
    assert {x[:2] for x in split | tile} == {t[:2] for t in f8_tiles.tiles()}
    # one product takes tiles of 8 rows up to 8 tokens only, whose weights are read by one workgroup alone
    assert {x[5:] for x in split if x[0] == 8} == {(1, 0), (1, 1), (0, 1)}
    for kernels in (split, tile):
        for x in kernels:
            if x[0] != 8:
                assert {x[:-2] + (once, grouped) for once in (0, 1) for grouped in (0, 1)} <= kernels
