"""A shape for every kernel that the block-scaled products and the norms choose from.
tests/test_fp8_host.py checks that each still takes the kernel named here, and
tests/test_gpu_fp8_kernels.py runs them."""

# waves, blocks of 16 weight rows, groups of 8 activation rows: (t, n, d)
DENSE_ROWS = {(4, 1, 1): (1, 300, 1040), (4, 1, 2): (9, 300, 1040), (4, 1, 4): (30, 300, 1040), (4, 1, 8): (64, 300, 1040),
              (4, 2, 1): (1, 8200, 400), (4, 2, 2): (16, 5130, 272), (4, 2, 4): (32, 5130, 272),
              (4, 2, 8): (64, 5130, 272), (4, 4, 4): (32, 10200, 272), (4, 4, 8): (50, 10200, 400),
              (8, 1, 1): (1, 300, 2064), (8, 1, 2): (9, 300, 2064), (8, 1, 4): (30, 300, 2064)}

# 64 x 128 tiles: whole, with every height of a part tile, one block and many
DENSE_64 = [(1473, 700, 272), (1488, 700, 272), (1489, 700, 272), (1504, 700, 272), (1505, 700, 272), (1520, 700, 272),
            (1521, 700, 272), (1535, 1003, 400), (1536, 1000, 128), (2500, 513, 1040), (1500, 400, 16)]
DENSE_256 = [(2049, 6001, 336), (2049, 6100, 400)]

# n, d, rows of each segment; few-row kernel of two and four waves, then tiles
LITTLE = [(7 * i) % 4 for i in range(300)]
GROUPED_ROWS = {(2, 2, 1): (1030, 272, LITTLE), (4, 2, 1): (130, 272, LITTLE[:60])}
GROUPED_64 = [(520, 272, [70, 3, 0, 64, 17, 33, 49])]
GROUPED_256 = [(640, 272, [97 + i for i in range(45)])]

# waves, groups of 8 elements a lane: (t, d)
NORMS = {(1, 1): (70, 504), (4, 1): (9, 1000), (8, 1): (5, 4000), (16, 1): (256, 5120), (4, 3): (257, 5120),
         (8, 2): (258, 7176), (8, 3): (4, 9000), (8, 4): (3, 14336), (16, 4): (3, 20000), (16, 8): (2, 40000)}
