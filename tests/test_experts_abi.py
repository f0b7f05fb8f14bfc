"""Refusals of the 8-bit linear layer and the expert-grouped products, before
any device work (safe without a GPU: nothing is launched), and their oracle."""
from __future__ import annotations

import re
from pathlib import Path

import numpy as np
import pytest

import oracle
import dequantize_mat_vec_amd as dmv
from dequantize_mat_vec_amd import _lib

HEADER = Path(__file__).resolve().parent.parent / "include" / "pesti.h"
FAKE = 0x100000   # 16-byte aligned, never dereferenced (calls are rejected)
F16, F32, I8, Q8 = 16, 17, 3, 0
MOST = 1 << 20


def test_constants_match_the_header():
    text = HEADER.read_text()
    for name, fid in list(dmv.VALUE_FORMAT_IDS.items()) + list(dmv.EXPERT_FORMAT_IDS.items()):
        assert re.search(rf"#define PESTI_FMT_{name.upper()} {fid}\b", text), name
    assert re.search(r"#define PESTI_MAX_TOKENS \(1 << 20\)", text)
    assert re.search(r"#define PESTI_MAX_EXPERTS 1024\b", text)


def test_quant_refusals():
    f = _lib.load().pesti_quant_i8token
    assert f(Q8, 4, 64, FAKE, FAKE, FAKE, None) == _lib.PESTI_ERR_SHAPE
    assert f(F16, -1, 64, FAKE, FAKE, FAKE, None) == _lib.PESTI_ERR_BATCH
    assert f(F16, MOST + 1, 64, FAKE, FAKE, FAKE, None) == _lib.PESTI_ERR_BATCH
    assert f(F16, 4, -32, FAKE, FAKE, FAKE, None) == _lib.PESTI_ERR_SHAPE
    assert f(F16, 4, 40, FAKE, FAKE, FAKE, None) == _lib.PESTI_ERR_SHAPE
    assert f(F16, 4, 32800, FAKE, FAKE, FAKE, None) == _lib.PESTI_ERR_SHAPE
    assert f(F32, 4, 64, None, FAKE, FAKE, None) == _lib.PESTI_ERR_NULL
    assert f(F32, 4, 64, FAKE, None, FAKE, None) == _lib.PESTI_ERR_NULL
    assert f(F32, 4, 64, FAKE, FAKE, None, None) == _lib.PESTI_ERR_NULL
    assert f(F32, 4, 64, FAKE + 8, FAKE, FAKE, None) == _lib.PESTI_ERR_ALIGN
    assert f(F32, 4, 64, FAKE, FAKE + 4, FAKE, None) == _lib.PESTI_ERR_ALIGN
    assert f(F32, 4, 64, FAKE, FAKE, FAKE + 2, None) == _lib.PESTI_ERR_ALIGN
    assert f(F32, 0, 64, None, None, None, None) == _lib.PESTI_OK


def test_gemm_i8_refusals():
    f = _lib.load().pesti_gemm_i8row_i8token

    def call(m=4, n=8, k=64, w=FAKE, ws=FAKE, x=FAKE, xs=FAKE, yf=F32, y=FAKE, b=None):
        return f(m, n, k, w, ws, x, xs, yf, y, b, None)

    assert call(yf=Q8) == _lib.PESTI_ERR_SHAPE
    assert call(m=-1) == _lib.PESTI_ERR_BATCH
    assert call(m=MOST + 1) == _lib.PESTI_ERR_BATCH
    assert call(n=-1) == _lib.PESTI_ERR_SHAPE
    for k in (-32, 40, 32800):
        assert call(k=k) == _lib.PESTI_ERR_SHAPE
    for name in ("w", "ws", "x", "xs", "y"):
        assert call(**{name: None}) == _lib.PESTI_ERR_NULL, name
    for name in ("w", "x", "y"):
        assert call(**{name: FAKE + 8}) == _lib.PESTI_ERR_ALIGN, name
    for name in ("ws", "xs", "b"):
        assert call(**{name: FAKE + 2}) == _lib.PESTI_ERR_ALIGN, name
    assert call(m=0, w=None, ws=None, x=None, xs=None, y=None) == _lib.PESTI_OK
    assert call(n=0, w=None, ws=None, x=None, xs=None, y=None) == _lib.PESTI_OK


def experts_call(gated, fmt=I8, rows=4, e=2, n=8, k=64, off=FAKE, w=FAKE, ws=FAKE, w2=FAKE, ws2=FAKE, t=4, x=FAKE,
                 xs=FAKE, at=None, yf=F32, y=FAKE, b=None):
    lib = _lib.load()
    if gated:
        return lib.pesti_gemm_experts_swiglu(fmt, rows, e, n, k, off, w, w2, ws, ws2, t, x, xs, at, yf, y, None)
    return lib.pesti_gemm_experts(fmt, rows, e, n, k, off, w, ws, t, x, xs, at, yf, y, b, None)


@pytest.mark.parametrize("gated", [False, True])
def test_experts_refusals(gated):
    def call(**kw):
        return experts_call(gated, **kw)

    for fmt in (Q8, F32, 99):
        assert call(fmt=fmt) == _lib.PESTI_ERR_SHAPE
    assert call(yf=I8) == _lib.PESTI_ERR_SHAPE
    assert call(n=-1) == _lib.PESTI_ERR_SHAPE
    for k in (-32, 40, 32800):
        assert call(k=k) == _lib.PESTI_ERR_SHAPE
    for e in (-1, 1025):
        assert call(e=e) == _lib.PESTI_ERR_SHAPE
    for kw in (dict(rows=-1), dict(rows=MOST + 1, t=MOST), dict(t=-1), dict(t=MOST + 1)):
        assert call(**kw) == _lib.PESTI_ERR_BATCH
    assert call(rows=5, t=4) == _lib.PESTI_ERR_BATCH        # no x_rows: row r of X itself
    # picked rows are addressed in 32 bits
    for fmt, t in ((F16, 1 << 16), (I8, 1 << 17)):
        assert call(fmt=fmt, k=32768, t=t, at=FAKE) == _lib.PESTI_ERR_SHAPE
    names = ["off", "w", "ws", "x", "xs", "y"] + (["w2", "ws2"] if gated else [])
    for name in names:
        assert call(**{name: None}) == _lib.PESTI_ERR_NULL, name
    for name in ["w", "x", "y"] + (["w2"] if gated else []):
        assert call(**{name: FAKE + 8}) == _lib.PESTI_ERR_ALIGN, name
    for name in ["off", "ws", "xs", "at"] + (["ws2"] if gated else ["b"]):
        assert call(**{name: FAKE + 2}) == _lib.PESTI_ERR_ALIGN, name
    empty = dict(off=None, w=None, ws=None, w2=None, ws2=None, x=None, xs=None, y=None)
    for kw in (dict(rows=0), dict(e=0), dict(n=0)):
        assert call(**kw, **empty) == _lib.PESTI_OK


@pytest.mark.parametrize("n", [1 << 31, 1 << 62, (1 << 63) - 1])
def test_columns_beyond_31_bits_are_refused(n):
    """Column tiles are numbered in 27 bits, and sums with so large a number would leave 64."""
    f = _lib.load().pesti_gemm_i8row_i8token
    assert f(4, n, 64, FAKE, FAKE, FAKE, FAKE, F32, FAKE, None, None) == _lib.PESTI_ERR_SHAPE
    for gated in (False, True):
        for rows in (4, 4096):
            assert experts_call(gated, n=n, rows=rows, t=rows) == _lib.PESTI_ERR_SHAPE


def test_binding_refuses_host_tensors_and_unknown_types():
    import torch
    with pytest.raises(ValueError):
        dmv.pesti_quant_i8token("f32", 1, 32, torch.zeros(32), FAKE, FAKE, stream=0)
    with pytest.raises(ValueError):   # a raw pointer says nothing about Y's type
        dmv.pesti_gemm_i8row_i8token(1, 32, 32, FAKE, FAKE, FAKE, FAKE, FAKE, stream=0)
    with pytest.raises(KeyError):
        dmv.pesti_gemm_experts("q4_k", 1, 1, 32, 32, FAKE, FAKE, 1, FAKE, FAKE, y_format="f32", stream=0)
    with pytest.raises(_lib.PestiError) as e:
        dmv.pesti_gemm_experts("i8row", 5, 1, 32, 32, FAKE, FAKE, 4, FAKE, FAKE, w_scales=FAKE, x_scales=FAKE,
                               y_format="f32", stream=0)
    assert e.value.status == _lib.PESTI_ERR_BATCH


def test_oracle_groups_rows():
    """Hand-worked: three experts, the middle one empty, one row behind the last."""
    w = np.array([[[1.0, 2.0]], [[3.0, 4.0]], [[5.0, 6.0]]])
    x = np.array([[1.0, 1.0], [0.0, 2.0]])
    y, size = oracle.gemm_experts([0, 2, 2, 3], w, x, 4, x_rows=[0, 1, 1, 0], bias=[[0.5], [0.0], [-1.0]])
    assert y[:3].tolist() == [[3.5], [4.5], [11.0]] and np.isnan(y[3, 0])
    assert size[:3].tolist() == [[3.5], [4.5], [13.0]]
    y, _ = oracle.gemm_experts([0, 1], w[:1], x, 1, x_rows=[7])
    assert y.tolist() == [[0.0]]
    assert oracle.expert_of_rows([-3, 2, 1, 9], 4).tolist() == [0, 2, 2, 2]
    y, size = oracle.gemm_i8([[1, -2]], [0.5], [[3, 4]], [2.0], [1.0])
    assert y.tolist() == [[-4.0]] and size.tolist() == [[6.0]]
