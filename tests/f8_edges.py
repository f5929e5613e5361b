"""Sizes of tests/test_f8_edges_gpu.py, which tests/test_f8_edges.py asks the launch's own rule about."""
# (E, M, N, K): more than 64 experts, 256 x 256 tiles
MANY = [(70, 12000, 2100, 1152), (72, 14896, 2302, 1176), (70, 6000, 4096, 144), (130, 20000, 1100, 520),
        (300, 30000, 1030, 272)]
# (tile, K): sums of more than 128 blocks, in the least sizes that take the tile
LONG = [(tile, K) for K in (16400, 24592, 33000) for tile in range(10)] + [(0, 131071), (1, 131071), (4, 131071)]
# (M, N, K) and (T, k, E, N, K) of the products that are captured, in the kernel of large tiles
GRAPH_DENSE = [(1024, 1024, 1152), (2048, 4096, 300), (4096, 4096, 1040)]
GRAPH_GROUPED = [(2048, 4, 16, 2048, 520), (1500, 3, 8, 1000, 300), (1700, 8, 70, 700, 1040)]
