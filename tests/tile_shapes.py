"""Shapes that reach every kernel behind the 8-bit and expert products, each
with the kernel that it takes: the GPU tests run them, and a test without a
GPU holds them against the library's own rule, so that another rule cannot
leave a kernel untested."""
from __future__ import annotations

FORMS = ("f16", "i8")

# Rows of an expert that end a tile of height h in every way: one row more than whole tiles, a whole tile, half
# a tile, one row more than half, none, one row alone, one row short.
def _ends(h):
    return [2 * h + 1, h, h // 2, h // 2 + 1, 0, 1, h - 1, 2 * h + h // 2, h + h // 2 + 1]


# (kernel, rows of each expert, columns, k): columns of the joined gate and up products are half as many.  More
# tiles than workgroups: each takes several, of different experts and heights.  K of one step, of a step and a
# quarter or more, and of many with the last one not full.
TILES = [(name, counts, n, k)
         for name, counts, n in (("256x256", 2 * _ends(256), 8001), ("128x256", 2 * _ends(128), 5003),
                                 ("128x128", 2 * _ends(128), 6001),
                                 ("64x128", 2 * (_ends(64)[1:] + [65, 40, 20, 35, 33, 48]), 7201))
         for k in (32, 160, 608)]
TILES += [("256x256", [400 + 3 * e for e in range(70)], 721, 32)]   # more experts than lanes

# dense 8-bit products: the last rows of Y are one alone, half a tile, one more
DENSE = [("256x256", 2817, 9001), ("256x256", 2944, 9000), ("256x256", 2945, 9001),
         ("128x256", 2305, 9001), ("128x256", 2368, 9001), ("128x256", 2369, 9000),
         ("128x128", 2177, 4096), ("128x128", 2240, 4097), ("128x128", 2241, 4097),
         ("64x128", 1665, 4864), ("64x128", 1696, 4863)]

# (kernel, rows of each expert or None for the dense call, columns, gated or not); each with both numbers of
# wavefronts
ROWS = [("rows 16", [3, 0, 16, 1, 17], 200, False), ("rows 16", [3, 0, 16, 1, 17], 201, True),
        ("rows 16", [i % 4 for i in range(70)], 72, False), ("rows 16", [i % 4 for i in range(70)], 71, True),
        ("rows 32", [100, 40, 0, 33, 31], 500, False), ("rows 32", [100, 40, 0, 33, 31], 499, True),
        ("rows 64", [200], 896, False), ("rows 64", [130, 65], 791, False),
        ("rows 64", None, 896, False), ("rows 64", None, 891, False)]
ROWS_DENSE_M = {896: 256, 891: 197}
SHORT_K, LONG_K = {"f16": (32, 928), "i8": (96, 1888)}, {"f16": (1056, 2464), "i8": (2080, 4864)}   # 2 and 4 wavefronts
