"""Infinite and NaN group scales of the 4-bit mat-vec: a row's scales reach that row alone, whichever way the work is
dealt out and wherever the row's last group ends within a chunk of 128 weights."""
from __future__ import annotations

import numpy as np
import pytest

import dequantize_mat_vec_amd as dmv
from gpu_util import announce, guarded_y, guards_intact, to_dev
from kv_reference import i4_matrix
from test_gpu_i4group import put, run

pytestmark = pytest.mark.gpu

# rows whose length is no multiple of 128, so that groups of a row's last chunk lie past its end: on the vector ALUs, a
# wavefront a tile, dealt out, in phases; rows shorter than a chunk
ENDS = [(1, 40, 928, 32), (2, 40, 2080, 64), (5, 4801, 800, 32), (8, 50003, 64, 32), (7, 60005, 32, 64), (5, 3101, 928, 64),
        (5, 2101, 2080, 64), (8, 1045, 8224, 32), (8, 1045, 8256, 64)]
VALUES = [np.inf, -np.inf, np.nan]


def rng_of(*key):
    return np.random.default_rng([74, *key])


def spoiled(m, value):
    """m with every scale of every third row `value`, and which rows those are."""
    packed, scales, zeros = m
    rows = np.arange(len(scales)) % 3 == 1
    scales = scales.copy()
    scales[rows] = value
    return (packed, scales, zeros), rows


@pytest.mark.parametrize("batch,out,inf,group", ENDS)
def test_a_scale_reaches_its_own_row_alone(batch, out, inf, group):
    announce(f"i4group scales {batch}x{out}x{inf} group {group}")
    rng = rng_of(1, out, inf)
    m = i4_matrix(rng, out, inf, group)
    x = rng.standard_normal((batch, inf)).astype(np.float32)
    bias = rng.standard_normal(out).astype(np.float32)
    want = run(m, out, inf, group, x, bias)
    assert np.isfinite(want).all()
    for value in VALUES:
        bad, rows = spoiled(m, value)
        y = run(bad, out, inf, group, x, bias)
        assert np.array_equal(y[:, ~rows], want[:, ~rows]), value
        assert not np.isfinite(y[:, rows]).any(), value


@pytest.mark.parametrize("batch,out,inf,group", [(1, 33, 928, 32), (2, 33, 2080, 64), (4, 9003, 800, 32), (5, 2500, 928, 64),
                                                 (8, 1045, 8224, 32)])
@pytest.mark.parametrize("which", ["gate", "up"])
def test_a_scale_reaches_its_own_row_alone_in_swiglu(batch, out, inf, group, which):
    announce(f"i4group swiglu scales {batch}x{out}x{inf} group {group} {which}")
    import torch
    rng = rng_of(2, out, inf)
    gate, up = (i4_matrix(rng, out, inf, group) for _ in range(2))
    x = to_dev(rng.standard_normal((batch, inf)).astype(np.float32))

    def swiglu(g, u):
        buf, h = guarded_y(batch * out)
        dmv.pesti_gemv_i4group_swiglu(out, inf, group, *put(g), *put(u), x, h, batch)
        torch.cuda.synchronize()
        assert guards_intact(buf, batch * out)
        return h.cpu().numpy().reshape(batch, out)

    want = swiglu(gate, up)
    assert np.isfinite(want).all()
    for value in VALUES:
        bad, rows = spoiled(gate if which == "gate" else up, value)
        h = swiglu(bad, up) if which == "gate" else swiglu(gate, bad)
        assert np.array_equal(h[:, ~rows], want[:, ~rows]), value


OWN = ENDS + [(1, 40, 896, 128), (2, 33, 96, 32), (5, 3101, 928, 32), (8, 4115, 4096, 64), (8, 1045, 8192, 128)]


@pytest.mark.parametrize("batch,out,inf,group", OWN)
def test_an_infinite_scale_gives_infinities(batch, out, inf, group):
    """Weights of one sign times positive x: an infinite scale of any one group is an infinite sum, of its sign."""
    announce(f"i4group infinite scale {batch}x{out}x{inf} group {group}")
    rng = rng_of(3, out, inf)
    packed, scales, zeros = i4_matrix(rng, out, inf, group)
    zeros[:] = 20   # every q - z is negative
    rows = np.arange(0, out, 3)
    at = rng.integers(0, scales.shape[1], len(rows))
    at[: len(rows) // 2] = 0
    sign = np.where(rng.random(len(rows)) < 0.5, -1.0, 1.0)
    scales[rows, at] = sign * np.inf
    for x in (rng.random((batch, inf)) + 0.1, np.ones((batch, inf))):   # (ones: nothing is left for a second part)
        y = run((packed, scales, zeros), out, inf, group, x.astype(np.float32))
        assert np.array_equal(y[:, rows], np.broadcast_to(-sign * np.inf, (batch, len(rows))))
        assert np.isfinite(np.delete(y, rows, 1)).all()


def test_an_infinite_scale_in_swiglu():
    announce("i4group infinite scale in swiglu")
    import torch
    for batch, out, inf, group in ((1, 33, 928, 32), (4, 9003, 800, 32), (5, 2500, 928, 64), (8, 1045, 8224, 32)):
        rng = rng_of(4, out, inf)
        gate, up = (i4_matrix(rng, out, inf, group) for _ in range(2))
        gate[0][:] |= 0x11
        gate[2][:], up[2][:] = 0, 20   # weights of gate are positive, those of up negative
        up[1][0::3, 0], gate[1][1::3, -1] = np.inf, np.inf
        x = to_dev((rng.random((batch, inf)) + 0.1).astype(np.float32))
        buf, h = guarded_y(batch * out)
        dmv.pesti_gemv_i4group_swiglu(out, inf, group, *put(gate), *put(up), x, h, batch)
        torch.cuda.synchronize()
        assert guards_intact(buf, batch * out)
        h = h.cpu().numpy().reshape(batch, out)
        assert np.all(h[:, 0::3] == -np.inf) and np.all(h[:, 1::3] == -np.inf) and np.isfinite(h[:, 2::3]).all()
