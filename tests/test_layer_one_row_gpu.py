"""qr_gemm_i8 in the kernels that test_layer_tiles_gpu.py does not run: those whose weights one row of tiles covers (they
are loaded past the caches), in every tile, and several rows of 128x64 and 64x32 tiles.  Sums of one stage (128 codes), of
fewer and of more stages than a ring holds or a workgroup has waves, whole and cut, each with ragged last tiles.  That each
size takes the tile it stands under is tested in test_layer_tile_choice.py.  Inputs, tolerances and the 64-bit reference are
those of test_layer_gpu.check_product."""
import pytest
import torch

from test_layer_gpu import check_product, qr  # noqa: F401  (qr: a fixture)

pytestmark = pytest.mark.gpu

# (tokens and channels of a tile, waves, one row of tiles or more): tokens, channels, stages
SIZES = {
    (16, 32, 4, 0, "one"): [(10, 4316, 1), (9, 4263, 2), (10, 4135, 3), (9, 4268, 4), (16, 4124, 5), (13, 4139, 11),
                            (10, 4167, 12), (11, 4206, 13), (13, 4142, 17), (9, 4245, 27), (14, 4274, 33), (12, 4430, 128)],
    (32, 32, 4, 0, "one"): [(17, 2289, 1), (27, 2101, 2), (32, 2058, 3), (25, 2117, 4), (22, 2060, 5), (19, 4167, 7),
                            (17, 4155, 8), (23, 4210, 9), (29, 4102, 13), (17, 4125, 19), (29, 4158, 33), (20, 4297, 128)],
    (64, 32, 4, 0, "one"): [(44, 4198, 11), (43, 4196, 12), (57, 4170, 13), (56, 4157, 17), (44, 4097, 27), (41, 4249, 100)],
    (64, 32, 4, 0, "more"): [(582, 421, 11), (611, 414, 12), (565, 470, 13), (599, 423, 17), (453, 563, 27), (543, 489, 128)],
    (64, 64, 4, 0, "one"): [(35, 8401, 33), (38, 8402, 48), (19, 8282, 64), (38, 8347, 100)],
    (64, 128, 2, 4, "one"): [(14, 17510, 1), (21, 16778, 2), (31, 16795, 4), (26, 17027, 5), (40, 16409, 6), (25, 16437, 7),
                             (29, 17163, 11)],
    (128, 64, 4, 2, "one"): [(72, 8404, 1), (72, 8767, 2), (81, 8566, 4), (70, 8546, 5), (73, 8703, 6), (70, 8470, 7),
                             (75, 8726, 11)],
    (128, 64, 4, 2, "more"): [(1617, 1163, 1), (1610, 1165, 2), (1609, 1177, 4), (1610, 1172, 5), (1615, 1153, 6),
                              (1602, 1158, 7), (1620, 1153, 11)],
    (128, 128, 2, 4, "one"): [(67, 16626, 1), (65, 18754, 2), (70, 17294, 3), (75, 16497, 4), (85, 17105, 5), (82, 16570, 6),
                              (67, 17525, 9)],
    (128, 256, 2, 4, "one"): [(17, 35658, 1), (20, 34902, 2), (20, 37698, 3), (9, 39271, 4), (9, 35594, 5), (20, 35561, 7)],
    (256, 256, 4, 2, "one"): [(138, 35273, 1), (133, 39471, 2), (137, 38044, 3), (154, 33430, 4), (177, 33178, 5)],
}


@pytest.mark.parametrize("tile", sorted(SIZES), ids=str)
@pytest.mark.parametrize("cut", [0, 5, 16, 127])
def test_rings(qr, tile, cut):  # noqa: F811
    g = torch.Generator(device="cuda").manual_seed(cut + 1)
    for i, (M, N, stages) in enumerate(SIZES[tile]):
        print("rings", tile, M, N, stages, cut, flush=True)
        check_product(qr, M, N, 128 * stages - cut, (torch.float16, torch.bfloat16)[i % 2], bool((i + cut) % 2), g)
