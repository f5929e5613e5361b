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
