"""The second binary16 parts of x, q and the softmax's weights, on operands long enough that a chain of float32 additions
may be off by more than they hold of a random value: here every value lies just short of the middle between two
binary16 numbers and all errors have one sign, so that a result of first parts alone is far outside the bound."""
from __future__ import annotations

import numpy as np
import pytest

from gpu_util import announce
from kv_reference import Cache, i4_matrix, i4_tolerance, i4_weights
from test_gpu_attention import attend
from test_gpu_i4group import run
from test_gpu_kv_cache import OnGpu

pytestmark = pytest.mark.gpu

BETWEEN = 1 + 2.0 ** -11 - 2.0 ** -16   # binary16 gives 1, a part in 2^11 too little


# dealt out, in phases, a wavefront a tile; rows of up to 32768 weights
@pytest.mark.parametrize("batch,out,inf,group", [(5, 4801, 800, 32), (8, 1045, 8224, 128), (8, 4115, 8192, 64), (3, 4115, 28704, 128),
                                                 (8, 1045, 32768, 32), (8, 32763, 2080, 64), (5, 2101, 16384, 256)])
def test_x_of_the_matrix_cores(batch, out, inf, group):
    announce(f"i4group second parts {batch}x{out}x{inf}")
    rng = np.random.default_rng([76, out, inf])
    packed, scales, zeros = m = i4_matrix(rng, out, inf, group)
    zeros[:] = 20   # weights of one sign
    x = (BETWEEN * 2.0 ** rng.integers(-3, 4, (batch, 1)) * np.ones((batch, inf))).astype(np.float32)
    y = run(m, out, inf, group, x)
    first, xd = x.astype(np.float16).astype(np.float64), x.astype(np.float64)
    for rows in np.array_split(np.arange(out), -(-out * inf // (1 << 24))):
        w = i4_weights(packed[rows], scales[rows], zeros[rows], inf, group)
        exact, tol = xd @ w.T, i4_tolerance(w, xd) + 2.0 ** -24 * np.abs(xd @ w.T)
        assert np.all(np.abs(first @ w.T - exact) > 2 * tol)
        assert np.all(np.abs(y[:, rows] - exact) <= tol)


def within(g, c, q, first):
    """attend() within the bound of the exact result, from which `first` (what first parts alone give) is far."""
    y = attend(g, 0, q, 1.0)
    exact, bound = c.attend(0, q, 1.0)
    tol = bound + 2.0 ** -24 * (np.abs(exact) + bound)
    assert np.all(np.abs(first - exact) > 2 * tol), float((np.abs(first - exact) / tol).min())
    assert np.all(np.abs(y - exact) <= tol), float((np.abs(y - exact) / tol).max())


LONG = [(64, 300), (64, 2000), (128, 9000), (64, 20000), (256, 9000), (32, 9000)]


def cache_of(fmt, d, n):
    """One sequence of n tokens, one KV head, K and V of zeros and (in 8 bits) scales of 2^-6."""
    c = Cache(np.random.default_rng([77, n]), fmt, 1, -(-n // 64) + 1, 64, 1, d, 1, -(-n // 64), [n])
    c.k[:], c.v[:] = 0, 0
    if fmt == "i8row":
        c.k_scales[:], c.v_scales[:] = 2.0 ** -6, 2.0 ** -6
    return c


def put(c, name, values):
    """values [tokens]: every dimension of the sequence's tokens."""
    t = np.arange(len(values))
    getattr(c, name)[0, c.table[0, t // c.page_size], 0, t % c.page_size] = (values if c.fmt == "f16" else values * 64)[:, None]


@pytest.mark.parametrize("fmt", ["f16", "i8row"])
@pytest.mark.parametrize("d,n", LONG)
def test_q(fmt, d, n):
    """Tokens of score 4 and few of score 8 that weigh as much together, V +-1: an error of the scores shifts the sum."""
    announce(f"attend second parts of q {fmt} d {d} {n} tokens")
    c = cache_of(fmt, d, n)
    high = np.zeros(n, bool)
    high[np.linspace(0, n - 1, round(n / np.exp(4))).astype(int)] = True
    put(c, "k", np.where(high, 1.0, 0.5))
    put(c, "v", np.where(high, 1.0, -1.0))
    q = np.full((1, 2, d), BETWEEN * 8 / d, np.float32)   # (d is a power of two)
    first, _ = c.attend(0, q.astype(np.float16), 1.0)
    within(OnGpu(c), c, q, first)


@pytest.mark.parametrize("fmt", ["f16", "i8row"])
@pytest.mark.parametrize("d,n", LONG)
def test_weights(fmt, d, n):
    """In every tile of 32 tokens one of the largest score; the others' weights lie between two binary16 numbers."""
    announce(f"attend second parts of the weights {fmt} d {d} {n} tokens")
    c = cache_of(fmt, d, n)
    high = np.arange(n) % 32 == 0
    put(c, "k", np.where(high, 1.0, 0.0))
    put(c, "v", np.where(high, 0.0, 1.0))
    gap = -np.log(BETWEEN / 2)   # a weight of BETWEEN / 2 of the largest
    q = np.full((1, 2, d), gap / d, np.float32)
    p = np.where(high, 1.0, BETWEEN / 2)
    first = np.full((1, 2, d), (0.5 * (~high).sum()) / p.sum())
    within(OnGpu(c), c, q, first)
