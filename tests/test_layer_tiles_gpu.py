"""qr_gemm_i8 at the edges of its rings of stages (128 codes each): sums of one stage, of fewer and of more stages than
a ring holds or a workgroup has waves, whole and cut, in every tile that the launch chooses, each with ragged last tiles.
Inputs, tolerances and the 64-bit reference are those of test_layer_gpu.check_product."""
import pytest
import torch

from test_layer_gpu import check_product, qr  # noqa: F401  (qr: a fixture)

pytestmark = pytest.mark.gpu

# tokens, channels, stages; the tile each list is for
SIZES = {
    "8x16": [(1, 33, s) for s in (1, 2, 4, 5, 8, 11, 12, 13, 24, 25)] + [(8, 50, 7), (5, 17, 128), (3, 4097, 33), (2, 4500, 40)],
    "8x16 of 8 waves": [(1, 33, s) for s in (33, 34, 39, 40, 41, 47, 48, 49, 64)] + [(8, 4095, 33), (7, 100, 129)],
    "16x16": [(9, 4, s) for s in (1, 2, 7, 8, 9, 15, 16, 17, 23, 24, 25)] + [(27, 35, 128)],
    "16x32": [(2050, 17, 1), (2121, 17, 2), (2071, 17, 3), (2055, 17, 4), (2049, 17, 5), (2116, 17, 12),
              (2095, 17, 13)],
    "32x32": [(4130, 4, 1), (4129, 4, 3), (4102, 4, 4), (4133, 4, 5), (4166, 4, 7), (4148, 4, 8), (4097, 4, 9)],
    "64x32": [(33, 4113, 12), (4138, 33, 13), (33, 4203, 17)],
    "64x64 of k_split": [(333, 2001, 33), (1001, 777, 40), (1001, 1013, 64)],
    "64x64 of k_tile": [(33, 4156, 1), (33, 4103, 2), (34, 4148, 3), (33, 4189, 4), (33, 4426, 5), (4177, 33, 6),
                        (4149, 34, 8)],
    "64x128 or 128x64": [(120, 9000, 1), (97, 9011, 4), (120, 9001, 5), (99, 9000, 6), (133, 5709, 1), (142, 5465, 2), (133, 5720, 4), (129, 5542, 5), (129, 5697, 6), (145, 5463, 7)],
    "64x128": [(273, 5511, 1), (262, 5681, 3), (258, 5798, 4), (258, 5896, 5), (262, 5971, 6)],
    "128x256": [(647, 5468, 1), (654, 5487, 2), (513, 6803, 3), (516, 6967, 4), (667, 5615, 6)],
    "128x128 of 3 rows of tiles": [(333, 8033, s) for s in (1, 3, 4, 5, 8, 9)],
    "256x256": [(4667, 1537, 1), (4869, 1542, 2), (1161, 6451, 3), (1290, 5895, 4)],
}


@pytest.mark.parametrize("tile", sorted(SIZES))
@pytest.mark.parametrize("cut", [0, 5, 16, 127])
def test_rings(qr, tile, cut):  # noqa: F811
    g = torch.Generator(device="cuda").manual_seed(cut)
    for i, (M, N, stages) in enumerate(SIZES[tile]):
        print("rings", tile, M, N, stages, cut, flush=True)
        check_product(qr, M, N, 128 * stages - cut, (torch.float16, torch.bfloat16)[i % 2], bool((i + cut) % 2), g)


def test_padding_does_not_matter(qr):  # noqa: F811
    """what the bytes of a row past K hold changes nothing"""
    g = torch.Generator(device="cuda").manual_seed(9)
    for M, N, K in ((1, 70, 129), (20, 33, 1000), (70, 4200, 250), (300, 5600, 33)):
        outs = []
        a = torch.randint(-128, 128, (M, K), generator=g, device="cuda", dtype=torch.int8)
        b = torch.randint(-128, 128, (N, K), generator=g, device="cuda", dtype=torch.int8)
        sa, sb = torch.rand(M, device="cuda"), torch.rand(N, device="cuda") / K
        for fill in (0, 127, -128):
            pa, pb = (torch.full((n, -(-K // 16) * 16), fill, dtype=torch.int8, device="cuda") for n in (M, N))
            pa[:, :K], pb[:, :K] = a, b
            c = torch.empty(M, N, dtype=torch.float16, device="cuda")
            qr.qr_gemm_i8(pa[:, :K], sa, pb[:, :K], sb, c)
            outs.append(c)
        torch.cuda.synchronize()
        assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2]), (M, N, K)
