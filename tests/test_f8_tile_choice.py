"""Which tile a size takes (tests/f8_tiles.py), on the host: every tile is taken by one product and by groups, and by
sums that end everywhere in its ring and in the parts in which scales come."""
import pytest

import f8_tiles

EDGES = [16, 128, 129, 256, 383, 384, 512, 640, 1023, 1024, 1040, 1152, 2048, 2049, 8192, 8200, 8320]


def test_every_tile_is_reached():
    one = {t for K in EDGES for t in f8_tiles.smallest(K, 0)}
    grouped = {t for K in EDGES for E in (1, 8, 70) for t in f8_tiles.smallest(K, E)}
    assert one == grouped == set(range(len(f8_tiles.tiles())))


@pytest.mark.parametrize("tile", range(10))
def test_edges_of_each_tile(tile):
    assert len(f8_tiles.tiles()) == 10
    found = [K for K in EDGES if tile in f8_tiles.smallest(K, 0) or tile in f8_tiles.smallest(K, 8)]
    assert any(K > 1024 for K in found)                       # scales in several parts
    rows, channels, stages, _ = f8_tiles.tiles()[tile]
    if (rows, channels) != (64, 128):                         # taken for sums of 2048 and more only
        assert any(K <= 128 * stages for K in found)          # a ring that is not filled


def test_small_batches_are_read_past_the_caches_only_once():
    """8 tokens and less take the 8-row tile"""
    sizes = [(0, M, N, K) for M in (1, 8) for N in (16, 300, 8192) for K in (64, 16384)]
    assert set(f8_tiles.choices(sizes)) == {0}
    assert 0 not in f8_tiles.choices([(0, 9, N, K) for N in (16, 300, 8192) for K in (64, 16384)])


def test_every_grid_fits_a_launch():
    """lanes are counted in 32 bits: tiles that would need more are not taken, and no tile where all would"""
    sizes = [(E, M, N, K) for E in (0, 1, 64, 1024) for M in (8, 512, 1024, 1 << 22) for K in (16, 8192)
             for N in (1 << 16, 1 << 18, 1 << 20, 1 << 22)]
    fits = {tile: 0 for tile in range(-1, 10)}
    for (E, M, N, _), tile in zip(sizes, f8_tiles.choices(sizes)):
        fits[tile] += 1
        some = min(E, M)
        for i, (rows, channels, _, threads) in enumerate(f8_tiles.with_threads()):
            tiles = -(-M // rows) if E == 0 else (M - some) // rows + some
            lanes = tiles * -(-N // channels) * threads
            if i == tile or (tile == -1 and i == 9):
                assert (lanes < 1 << 32) == (tile >= 0), (E, M, N, tile, lanes)
    assert fits[-1] > 0 and fits[9] > 0
