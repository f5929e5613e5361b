"""Sizes of tests/test_f8_edges_gpu.py, which tests/test_f8_edges.py asks the launch's own rule about."""
# (E, M, N, K): more than 64 experts, 256 x 256 tiles
MANY = [(70, 12000, 2100, 1152), (72, 14896, 2302, 1176), (70, 6000, 4096, 144), (130, 20000, 1100, 520),
        (300, 30000, 1030, 272)]
# (tile, K): sums of more than 128 blocks, in the least sizes that take the tile
LONG = [(tile, K) for K in (16400, 24592, 33000) for tile in range(10)] + [(0, 131071), (1, 131071), (4, 131071)]
# (M, N, K) and (T, k, E, N, K) of the products that are captured, in the kernel of large tiles
GRAPH_DENSE = [(1024, 1024, 1152), (2048, 4096, 300), (4096, 4096, 1040)]
GRAPH_GROUPED = [(2048, 4, 16, 2048, 520), (1500, 3, 8, 1000, 300), (1700, 8, 70, 700, 1040)]
# (T, E, k) that reach every kernel of the router
ROUTES = [(1, 300, 8), (16, 512, 32), (17, 512, 8), (64, 257, 5), (64, 512, 32), (65, 512, 32), (65, 300, 1), (130, 300, 18),
          (32, 64, 8), (33, 60, 3), (65, 33, 32), (16, 128, 9), (17, 100, 2), (66, 127, 31), (16, 256, 8), (17, 200, 4),
          (127, 250, 17), (5, 1000, 32), (65, 513, 3)]


def kernel_of_route(T, E):
    """lanes to a token, logits to a lane, lanes of a workgroup, whether it is the only one"""
    G, V = ((8, 8) if E <= 64 else (16, 8) if E <= 128 else (16, 16) if E <= 256 else (64, 16) if E > 512 else
            (64, 8) if T <= 16 else (16, 32))
    return G, V, 256 if T <= 64 and E <= 256 and T * G <= 256 else 1024, int(T <= 64)
