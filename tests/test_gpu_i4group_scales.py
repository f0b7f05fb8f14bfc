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
