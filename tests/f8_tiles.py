"""Sizes that take a given tile of the products in 8-bit floating point, found by asking the launch's own rule."""
import functools
import os
import subprocess
import tempfile

HERE = os.path.dirname(os.path.abspath(__file__))


@functools.lru_cache(None)
def program():
    exe = os.path.join(tempfile.mkdtemp(), "f8_tiles_print")
    subprocess.run(["g++", "-std=c++17", "-O1", "-o", exe, os.path.join(HERE, "f8_tiles_print.cpp")], check=True)
    return exe


@functools.lru_cache(None)
def with_threads():
    """(rows, channels, stages of a ring, threads of a workgroup)"""
    out = subprocess.run([program(), "list"], capture_output=True, text=True, check=True).stdout
    return [tuple(map(int, line.split()))[:3] + (int(line.split()[4]),) for line in out.splitlines()]


@functools.lru_cache(None)
def tiles():
    """(rows, channels, stages of a ring, waves along the channels or 0)"""
    out = subprocess.run([program(), "list"], capture_output=True, text=True, check=True).stdout
    return [tuple(map(int, line.split()))[:4] for line in out.splitlines()]


def choices(sizes):
    text = "".join("%d %d %d %d\n" % s for s in sizes)
    out = subprocess.run([program()], input=text, capture_output=True, text=True, check=True).stdout
    return list(map(int, out.split()))


@functools.lru_cache(None)
def smallest(K, E):
    """{tile: (M, N)} of the least M * N that takes it, for sums of K and E experts (0: one product)"""
    Ms = sorted({m + d for m in (1, 2, 4, 8, 16, 24, 32, 48, 64, 96, 128, 192, 256, 384, 512, 768, 1024, 1536, 2048, 3000,
                                 4096) for d in (0, 1)})
    Ns = sorted({n + d for n in (16, 48, 64, 128, 256, 384, 512, 1024, 2048, 4096, 8192, 16384) for d in (0, 5)})
    sizes = sorted(((E, M, N, K) for M in Ms for N in Ns), key=lambda s: s[1] * s[2])
    found = {}
    for (_, M, N, _), tile in zip(sizes, choices(sizes)):
        found.setdefault(tile, (M, N))
    return found
