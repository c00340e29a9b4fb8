"""Sizes (M, N, K) at which the MX4 products take each of their kernels on 256
compute units.  A CPU test asserts that the library plans them so; GPU tests
run them.

A tile over `groups` groups of waves steps through rounds of 4 * groups tiles
of 128 k; a size in ROUNDS has at least three whole rounds and a part of one,
so that the ring of stages, the two buffers of scales and the counted waits
come round, and every group has tiles.  STAY adds the other kind of result
stores (large outputs of rows that are no whole lines, short k)."""

CUS = 256

# Rows, columns and groups of the output tiles.
TILES = {
    "w4": [(16, 64, 8), (32, 64, 4), (64, 64, 4), (64, 128, 2), (32, 256, 1), (64, 256, 1),
           (128, 256, 1), (256, 256, 1)],
    "w2": [(16, 64, 8), (32, 64, 4), (32, 128, 4), (64, 128, 2), (32, 256, 1), (64, 256, 1),
           (128, 256, 1)],
}

# In the order of TILES, then neighbours of projection sizes.
ROUNDS = {
    "w4": [(33, 36, 13127), (2057, 71, 6821), (34, 8508, 6700), (5443, 129, 3597),
           (193, 8223, 1655), (5508, 259, 1626), (5690, 513, 1609), (5441, 1401, 2110),
           (511, 2561, 6900), (513, 13825, 2600), (257, 13823, 5200)],
    "w2": [(35, 35, 12809), (4125, 34, 6959), (4187, 68, 6915), (5777, 132, 3587),
           (195, 8693, 1601), (5448, 259, 1603), (5453, 670, 2185),
           (511, 2561, 6900), (513, 13825, 2600), (257, 13823, 5200)],
}

# Results of every output selection stay in the caches.
STAY = {
    "w4": [(691, 22091, 100), (268, 47487, 1542), (374, 34105, 1545), (1486, 8472, 1543)],
    "w2": [(277, 53489, 73), (259, 48773, 1544), (9409, 1339, 1540)],
}

# Of the weight stream: rows of its form and waves to a strip, three quads of
# tiles or more to each wave.
STREAM = {
    "w4": [(1, 100, 13000), (1, 4200, 5200), (13, 90, 8300), (9, 4200, 3500), (16, 16500, 1700),
           (32, 70, 5200), (29, 4200, 3500), (17, 8300, 1700)],
    "w2": [(1, 100, 13000), (1, 8300, 5200), (13, 90, 8300), (9, 8300, 3500), (16, 33000, 1700),
           (32, 70, 5200), (29, 8300, 3500), (17, 16500, 1700)],
}
STREAM_FORMS = [(1, 8), (1, 3), (16, 5), (16, 2), (16, 1), (32, 3), (32, 2), (32, 1)]
