"""The kernel that each shape of the GPU tests takes, by the library's own
rule: every kernel is reached, and the tile kernels with several tiles for a
workgroup."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle
import tile_choice as choice
import tile_reference as ref
import tile_shapes as shapes

LEAD_AND_BEHIND = 3   # rows of Y that belong to no expert


@pytest.mark.parametrize("form", shapes.FORMS)
@pytest.mark.parametrize("gated", [False, True])
def test_expert_shapes_take_the_tiles_that_they_name(gated, form):
    reached = set()
    for name, counts, n, k in shapes.TILES:
        n = n // 2 if gated else n
        assert choice.kernel(sum(counts) + LEAD_AND_BEHIND, n, k, form, len(counts), gated) == name
        tiles, workgroups = choice.tiles_and_workgroups(name, counts, n, len(counts), gated)
        assert tiles > workgroups, (name, counts, n)
        reached.add(name)
    assert reached == set(choice.NAMES[3:])


def test_dense_shapes_take_the_tiles_that_they_name():
    ends = {}
    for name, m, n in shapes.DENSE:
        assert choice.kernel(m, n, 96, "i8") == name
        tiles, workgroups = choice.tiles_and_workgroups(name, [m], n, 0)
        assert tiles > workgroups, (name, m, n)
        height = int(name.split("x")[0])
        ends.setdefault(name, set()).add((m % height) / height if m % height != 1 else 0.0)
    assert set(ends) == set(choice.NAMES[3:])
    for name, e in ends.items():
        assert {0.0, 0.5} <= e, name   # one row alone, half a tile


def test_few_rows_take_the_rows_kernels_that_they_name():
    reached = set()
    for name, counts, n, gated in shapes.ROWS:
        for form in shapes.FORMS if counts else ("i8",):
            for ks, wavefronts in ((shapes.SHORT_K, 2), (shapes.LONG_K, 4)):
                for k in ks[form]:
                    rows, e = (sum(counts) + LEAD_AND_BEHIND, len(counts)) if counts else (shapes.ROWS_DENSE_M[n], 0)
                    assert choice.kernel(rows, n, k, form, e, gated) == name, (rows, n, k, form, e, gated)
                    assert choice.wavefronts(k, form) == wavefronts
                    reached.add((name, wavefronts, form, gated))
    want = {(name, w, form, gated) for name in choice.NAMES[:3] for w in (2, 4) for form in shapes.FORMS for gated in (False, True)
            if not (gated and name == "rows 64")}   # not built
    assert reached == want


def test_rows_64_is_never_taken_for_joined_products():
    for experts in (0, 1, 2, 8, 64):
        for rows in list(range(1, 300)) + [1000, 4096]:
            for n in (1, 16, 100, 896, 2304, 4864):
                for k in (32, 896, 4864):
                    assert choice.kernel(rows, n, k, "f16", experts, True) != "rows 64"


@pytest.mark.parametrize("form", shapes.FORMS)
def test_reference_equals_the_oracle(form):
    """The torch reference of the GPU tests against the numpy oracle, bit for bit but for the order of a sum."""
    rng = np.random.default_rng(1)
    offsets, at = [1, 4, 4, 9], rng.integers(-1, 8, size=11).astype(np.int32)
    if form == "f16":
        x, xs, w, ws = rng.standard_normal((7, 32)).astype(np.float16), None, rng.standard_normal((3, 5, 32)).astype(np.float16), None
    else:
        x, w = (rng.integers(-128, 128, size=s).astype(np.int8) for s in ((7, 32), (3, 5, 32)))
        xs, ws = (rng.random(s).astype(np.float32) for s in (7, (3, 5)))
    bias = rng.standard_normal((3, 5)).astype(np.float32)

    def t(a):
        return None if a is None else torch.from_numpy(a)
    y, size = ref.grouped(offsets, t(w), t(x), t(at), t(bias), t(ws), t(xs))
    want, magnitude = oracle.gemm_experts(offsets, w, x, 11, at, bias, ws, xs)
    if ws is not None:   # exact sums: errors are relative to the product itself
        p, _ = oracle.gemm_experts(offsets, w, x, 11, at, None, ws, xs)
        magnitude = np.abs(p) + np.abs(want - p)
    np.testing.assert_allclose(y.numpy(), want, rtol=0, atol=1e-12 * np.nanmax(np.abs(want)), equal_nan=True)
    np.testing.assert_allclose(size.numpy(), magnitude, rtol=1e-9, atol=1e-9, equal_nan=True)
    assert np.isnan(want[0]).all() and np.isnan(want[9:]).all() and not np.isnan(want[1:9]).any()
