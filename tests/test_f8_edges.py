"""The sizes of the GPU tests of the products' tiles do run what they are meant to (no GPU needed)."""
import f8_tiles
from f8_edges import GRAPH_DENSE, GRAPH_GROUPED, LONG, MANY
from test_f8_tile_choice import EDGES


def test_every_tile_has_a_size_in_the_tests():
    """of test_f8_tiles_gpu.py, which passes over what has none"""
    without = [(tile, E) for E in (0, 1, 8, 70) for tile in range(10)
               if not any(tile in f8_tiles.smallest(K, E) for K in EDGES)]
    assert without == [(9, 70)]                      # MANY instead


def test_many_experts_in_large_tiles():
    assert {f8_tiles.tiles()[t][:2] for t in f8_tiles.choices(MANY)} == {(256, 256)}
    assert all(E > 64 for E, *_ in MANY) and any(E > 128 for E, *_ in MANY)


def test_long_sums_in_every_tile():
    assert all(K > 128 * 128 for _, K in LONG) and {tile for tile, _ in LONG} == set(range(10))
    for tile, K in LONG:
        assert tile in f8_tiles.smallest(K, 0) and tile in f8_tiles.smallest(K, 8), (tile, K)


def test_captured_products_take_large_tiles():
    taken = [f8_tiles.tiles()[t] for t in f8_tiles.choices([(0, *s) for s in GRAPH_DENSE]
                                                           + [(E, T * k, N, K) for T, k, E, N, K in GRAPH_GROUPED])]
    assert all(waves != 0 for *_, waves in taken)    # k_tile_f8
    assert (256, 256) in {t[:2] for t in taken[:3]} and (256, 256) in {t[:2] for t in taken[3:]}
