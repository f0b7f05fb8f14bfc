"""Infinities and NaN of V in a part of a sequence that the others outweigh: the join keeps them, as a sequence of one
part does."""
from __future__ import annotations

import numpy as np
import pytest

from gpu_util import announce
from kv_reference import Cache
from test_gpu_attention import attend
from test_gpu_kv_cache import OnGpu

pytestmark = pytest.mark.gpu

# one part; up to eight, joined by threads; more, joined by workgroups of 32, 64 and 128 dimensions
LENGTHS = [(64, 300), (64, 2000), (64, 9000), (64, 50000), (128, 2000), (128, 5000), (128, 20000), (32, 60000)]


def cache_of(fmt, d, longest, low):
    """One KV head whose first quarter of tokens score `low`, the others 300, for a q of 1 in dimension 0."""
    rng = np.random.default_rng([75, d, longest])
    page = 64
    c = Cache(rng, fmt, 1, -(-longest // page) + 1, page, 1, d, 1, -(-longest // page), [longest], shuffle=False)
    early = (np.arange(c.pages * page) < longest // 4).reshape(c.pages, page)
    c.k[:] = 0
    if fmt == "f16":
        c.k[0, :, 0, :, 0] = np.where(early, low, 300)
    else:
        c.k[0, :, 0, :, 0] = np.where(early, 0 if low == 0 else -127, 100)
        c.k_scales[:] = 3.0
        c.k_scales[0, :, 0][early] = np.inf if low == -np.inf else 3.0
    return c


def query(d):
    q = np.zeros((1, 3, d), np.float32)
    q[:, :, 0] = 1.0
    return q


@pytest.mark.parametrize("fmt", ["f16", "i8row"])
@pytest.mark.parametrize("d,longest", LENGTHS)
@pytest.mark.parametrize("low", [0.0, -np.inf])
def test_values_of_an_outweighed_part(d, longest, low, fmt):
    announce(f"attend outweighed part {fmt} d {d} {longest} tokens scores {low}")
    c = cache_of(fmt, d, longest, low)
    plain = attend(OnGpu(c), 0, query(d), 1.0)
    assert np.isfinite(plain).all()
    t = longest // 9
    for value in (np.nan, np.inf, -np.inf):
        bad = cache_of(fmt, d, longest, low)
        if fmt == "f16":
            bad.v[0, t // 64, 0, t % 64, 20] = value
            hit = np.arange(d) == 20
        else:
            bad.v[0, t // 64, 0, t % 64] = 5
            bad.v_scales[0, t // 64, 0, t % 64] = value   # of a row that was not finite: NaN of every dimension
            hit = np.ones(d, bool)
        y = attend(OnGpu(bad), 0, query(d), 1.0)
        assert not np.isfinite(y[:, :, hit]).any(), value
        assert np.array_equal(y[:, :, ~hit], plain[:, :, ~hit]), value


@pytest.mark.parametrize("d,longest", LENGTHS)
def test_parts_without_tokens_count_for_nothing(d, longest):
    """A bound far above the length leaves most parts empty, of which the workspace holds NaN."""
    announce(f"attend empty parts d {d} {longest} tokens")
    c = cache_of("f16", d, longest, 0.0)
    c.lengths[0] = 40
    y = attend(OnGpu(c), 0, query(d), 1.0, max_length=longest)
    c.lengths[0] = 0
    assert np.isfinite(y).all() and not attend(OnGpu(c), 0, query(d), 1.0, max_length=longest).any()
