"""Scores of any size: where float32's neighbours lie further apart than the softmax's weights reach, the largest tokens
take all of the sum."""
from __future__ import annotations

import numpy as np
import pytest

from gpu_util import announce
from kv_reference import Cache
from test_gpu_attention import attend
from test_gpu_kv_cache import OnGpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["f16", "i8row"])
@pytest.mark.parametrize("d,longest", [(64, 40), (64, 300), (64, 2000), (128, 9000), (32, 30000)])
def test_scores_of_every_size(fmt, d, longest):
    announce(f"attend large scores {fmt} d {d} {longest} tokens")
    rng = np.random.default_rng([78, d, longest])
    c = Cache(rng, fmt, 1, -(-longest // 32) + 1, 32, 1, d, 1, -(-longest // 32), [longest])
    if fmt == "i8row":
        c.k_scales[:] = 1.0
    # dimension 0 is the score: 100 for two tokens, 0 for two others, 25 to 75 for the rest
    key = rng.integers(25, 76, longest).astype(float)
    ends = {1.0: [longest // 5, longest - 2], -1.0: [longest // 3, longest // 2]}
    key[ends[1.0]], key[ends[-1.0]] = 100, 0
    t = np.arange(longest)
    c.k[:] = 0
    c.k[0, c.table[0, t // 32], 0, t % 32, 0] = key
    v, _ = c.rows("v", 0, 0, 0)
    g = OnGpu(c)
    for power in range(4, 110, 3):
        for sign in (1.0, -1.0):
            q = np.zeros((1, 3, d), np.float32)
            q[0, :, 0] = sign * 2.0 ** power * np.array([1.0, 1.37, 1.9])
            y = attend(g, 0, q, 1.0)
            want = v[ends[sign]].mean(0)
            # the others are 16 * 25 or more below: nothing.  Two equal weights, their sum and quotient: a few roundings
            assert np.all(np.abs(y[0] - want) <= 2.0 ** -21 * np.abs(v[ends[sign]]).mean(0)), (power, sign)
