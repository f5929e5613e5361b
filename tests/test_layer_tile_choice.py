"""The tile that qr_gemm_i8 takes for a size (csrc/qr_gemm_tiles.h, the rule that the launch uses, compiled here for the
host): the sizes of the GPU tests run the tiles they stand under, and every kernel that some size takes is among them."""
import os
import subprocess

import pytest

import test_layer_one_row_gpu
import test_layer_tiles_gpu

TESTS = os.path.dirname(os.path.abspath(__file__))
CUTS = (0, 5, 16, 127)


@pytest.fixture(scope="module")
def choose(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("tiles") / "print")
    subprocess.run(["g++", "-O1", "-Wall", "-Werror", "-std=c++17", os.path.join(TESTS, "gemm_tiles_print.cpp"), "-o", exe],
                   check=True)

    def choose(sizes):
        """(tokens, channels, waves, waves, one row of tiles or more) of each size"""
        out = subprocess.run([exe], input="".join("%d %d %d\n" % s for s in sizes), capture_output=True, text=True,
                             check=True).stdout.split("\n")[:-1]
        rows = [[int(x) for x in line.split()] for line in out]
        assert len(rows) == len(sizes)
        return [tuple(r[1:5]) + ("one" if r[6] == 1 else "more",) for r in rows]
    return choose


def cut_sizes(sizes):
    return [(M, N, 128 * stages - cut) for cut in CUTS for M, N, stages in sizes]


@pytest.mark.parametrize("tile", sorted(test_layer_one_row_gpu.SIZES), ids=str)
def test_sizes_take_their_tile(choose, tile):
    sizes = cut_sizes(test_layer_one_row_gpu.SIZES[tile])
    for size, got in zip(sizes, choose(sizes)):
        assert got == tile, size


# the tiles of each list of test_layer_tiles_gpu.py
LISTS = {
    "8x16": [(8, 16, 4, 0), (8, 16, 8, 0)], "8x16 of 8 waves": [(8, 16, 8, 0)], "16x16": [(16, 16, 8, 0)],
    "16x32": [(16, 32, 4, 0)], "32x32": [(32, 32, 4, 0)], "64x32": [(64, 32, 4, 0)],
    "64x64 of k_split": [(64, 64, 4, 0)], "64x64 of k_tile": [(64, 64, 2, 2)],
    "64x128 or 128x64": [(64, 128, 2, 4), (128, 64, 4, 2)], "64x128": [(64, 128, 2, 4)],
    "128x256": [(128, 256, 2, 4)], "128x128 of 3 rows of tiles": [(128, 128, 2, 4)], "256x256": [(256, 256, 4, 2)],
}


@pytest.mark.parametrize("label", sorted(LISTS))
def test_the_other_lists_take_theirs(choose, label):
    sizes = cut_sizes(test_layer_tiles_gpu.SIZES[label])
    for size, got in zip(sizes, choose(sizes)):
        assert got[:4] in LISTS[label], size


def test_every_kernel_that_a_size_takes_is_run(choose):
    run = set(test_layer_one_row_gpu.SIZES)
    for sizes in test_layer_tiles_gpu.SIZES.values():
        run |= set(choose(cut_sizes(sizes)))
    powers = [round(2 ** (x / 3)) for x in range(67)]
    tokens = [m for m in powers if m <= 16384] + [9, 17, 33, 48, 65, 100, 129, 200]
    codes = [1, 129, 512, 1000, 2048, 4096, 16384, 131071]
    sizes = [(M, N, K) for M in tokens for N in powers for K in codes]
    taken = {}
    for size, got in zip(sizes, choose(sizes)):
        taken.setdefault(got, size)
    missing = {tile: size for tile, size in taken.items() if tile not in run}
    assert not missing, missing
    assert len(taken) == 24, sorted(taken)         # 11 tiles of either kind, and two of up to 8 tokens


def test_tiles_of_8_tokens_are_one_row(choose):
    """the launch has these two only as kernels of one row of tiles"""
    sizes = [(M, N, K) for M in range(1, 70) for N in (1, 300, 4096, 4097, 1 << 20) for K in (1, 4095, 4096, 131071)]
    for size, got in zip(sizes, choose(sizes)):
        assert (got[0] == 8) == (size[0] <= 8) and (got[0] != 8 or got[4] == "one"), size
