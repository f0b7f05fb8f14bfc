"""A workspace of the attention sized for the most rows and the longest bound serves every smaller call (host code only)."""
from __future__ import annotations

import numpy as np
import pytest

from test_kv_abi import FAKE, WORKSPACE, addr, attend, cache, lib, table

LENGTHS = sorted({1, 31, 32, 33, 97, 512, 700, 768, 1000, 1500, 2047, 2048, 2049, 4096, 8191, 8192, 8193, 16384, 32767, 32768, 32769, 32800,
                  40000, 60000, 65536, 100000, 131071, 1 << 20, 1 << 30} | {128 * n for n in range(1, 260, 7)} | {256 * n for n in range(1, 260, 11)})
ROWS = [1, 2, 3, 4, 5, 7, 8, 12, 16, 23, 31, 32, 33, 48, 63, 64, 65, 100, 128, 255, 256, 300, 1000, 4096]
SHAPES = [(8, 32, 128), (1, 4, 128), (2, 14, 64), (1, 8, 32), (4, 16, 256), (12, 12, 64), (1, 40, 128), (1, 71, 64), (128, 128, 96)]


def size(c, rows, heads, longest):
    return lib().pesti_attn_paged_workspace_bytes(addr(c), rows, heads, longest)


@pytest.mark.parametrize("kv,heads,d", SHAPES)
def test_sizes_grow_with_rows_and_lengths(kv, heads, d):
    c = cache(kv_heads=kv, head_dim=d)
    sizes = np.array([[size(c, r, heads, n) for n in LENGTHS] for r in ROWS])
    assert (sizes >= 0).all() and (np.diff(sizes, axis=0) >= 0).all() and (np.diff(sizes, axis=1) >= 0).all()


@pytest.mark.parametrize("kv,heads,d", SHAPES)
def test_one_size_serves_every_smaller_call(kv, heads, d):
    import torch
    if torch.cuda.is_available():
        pytest.skip("calls that pass every check would be launched")
    c, t = cache(kv_heads=kv, head_dim=d), table(seqs=4096, width=1 << 20)

    def short(rows, longest, held):
        # (an unaligned workspace: refused for its size first)
        return attend(c, t, rows=rows, heads=heads, stride=heads * d, most=longest, ws=FAKE + 4, ws_bytes=held) == WORKSPACE

    for rows, longest in ((8, 1500), (64, 1500), (33, 8192), (1, 131071), (300, 131071), (2, 60000)):
        held = size(c, rows, heads, longest)
        tight = held == 0
        for r in (r for r in ROWS if r <= rows):
            for n in (n for n in LENGTHS + [longest] if n <= longest):
                assert not short(r, n, held), (rows, longest, r, n)
        # and no more than one of them needs
        for r in range(1, rows + 1):
            tight = tight or any(short(r, n, held - 1) for n in LENGTHS + [longest] + [128 * (256 // max(1, r * kv * k)) for k in (1, 2, 3, 5, 9)]
                                 if 1 <= n <= longest)
        assert tight, (rows, longest)
