"""Sizes at which the products with 4-bit weights (M, N, K) and the mixture of
experts (M, H, I, E, top_k) take each of their kernels on 256 compute units.
A CPU test asserts that the library plans them so; GPU tests run them."""

CUS = 256

# By w4a8_plan's (kernel, rows, groups, parts > 1), for groups of every length.  Of
# each kind one at least has several tiles a wave, and one ends inside a tile.
W4 = {
    (1, 1, 8, False): [(1, 100, 12800), (1, 40, 33000), (1, 17, 66001)],
    (1, 1, 4, False): [(1, 8300, 5201)],
    (2, 16, 4, True): [(2, 900, 13000), (9, 900, 6001)],
    (2, 16, 4, False): [(16, 8300, 5200), (9, 8300, 130)],
    (2, 16, 2, False): [(13, 16500, 3001)],
    (2, 32, 4, True): [(20, 500, 9000)],
    (2, 32, 4, False): [(32, 8300, 2001), (20, 8300, 257)],
    (2, 32, 2, True): [(17, 5200, 10201)],
    (2, 32, 2, False): [(32, 16500, 2000)],
    (2, 48, 2, True): [(48, 500, 9001)],
    (2, 48, 2, False): [(40, 8300, 2000), (33, 8300, 31)],
    (2, 64, 2, True): [(50, 700, 12001)],
    (2, 64, 2, False): [(64, 8300, 2000), (49, 8300, 65)],
    (3, 16, 8, False): [(2, 900, 6016), (16, 4000, 2049), (13, 5000, 1000), (7, 33, 4095)],
    (3, 32, 8, False): [(20, 500, 4000), (32, 100, 2047)],
    (3, 48, 8, False): [(40, 700, 1304), (33, 17, 1023)],
    (3, 64, 8, False): [(64, 900, 2000), (50, 31, 1023)],
    (3, 64, 3, False): [(64, 100, 300)],
}

# By moe_plan's (kernel, up, down).
MOE = {
    (1, 1, 1): [(1, 640, 1000, 64, 8), (2, 1300, 2001, 6, 3), (40, 100, 130, 5, 2)],
    (2, 1, 1): [(5, 1300, 4001, 6, 3), (1, 40, 3500, 16, 16)],
    (2, 2, 2): [(64, 1300, 1500, 64, 6)],
}
