"""Rows of K, V or q that a tensor does not have are refused, though its memory goes on behind them (no GPU needed)."""
from __future__ import annotations

import pytest

import dequantize_mat_vec_amd as dmv
from test_experts_types import DeviceTensor
from test_kv_abi import Rows


class Shaped(Rows):
    """A view of that shape and strides into a large memory."""

    def __init__(self, dtype, shape, strides):
        super().__init__(dtype, 1, 1)
        self.shape, self.strides, self.held = shape, strides, 1 << 20

    def stride(self):
        return self.strides


def calls():
    import torch
    f16, i32 = torch.float16, torch.int32
    t = DeviceTensor
    c = dmv.kv_cache("f16", 2, 8, 16, 2, 64, t(f16, 32768), t(f16, 32768))
    tab = dmv.kv_table(t(i32, 12), t(i32, 4), None, 4, 3)

    def append(k, rows=3, stride=None):   # layer 2 of two: what passes is refused by the library
        return dmv.pesti_cache_append(c, tab, 2, rows, k, k, stride=stride, stream=0)

    def attend(q, rows=3, stride=None):
        return dmv.pesti_attn_paged(c, tab, 2, rows, 2, q, t(torch.float32, 128 * rows), 1.0, q_stride=stride, workspace_bytes=0, stream=0)
    return append, attend


# (shape, strides, rows, stride): a row is 128 values
FIT = [((3, 128), (128, 1), 3, None), ((3, 128), (400, 1), 3, None), ((3, 400), (400, 1), 3, 400), ((3, 2, 64), (128, 64, 1), 3, None),
       ((6, 64), (64, 1), 3, 128), ((384,), (1,), 3, 128), ((1, 128), (7, 1), 1, None), ((5, 128), (128, 1), 3, None), ((0, 128), (128, 1), 0, None)]
SHORT = [((3, 64), (400, 1), 3, None), ((3, 64), (400, 1), 3, 400), ((2, 128), (400, 1), 3, 400), ((2, 128), (128, 1), 3, None),
         ((1, 64), (128, 1), 1, None), ((383,), (1,), 3, 128), ((3, 1, 64), (128, 64, 1), 3, None), ((0, 128), (128, 1), 1, None)]


@pytest.mark.parametrize("shape,strides,rows,stride", FIT)
def test_rows_that_are_there(shape, strides, rows, stride):
    import torch
    for call in calls():
        with pytest.raises(dmv.PestiError):
            call(Shaped(torch.float16, shape, strides), rows, stride)


@pytest.mark.parametrize("shape,strides,rows,stride", SHORT)
def test_rows_that_are_not_there(shape, strides, rows, stride):
    import torch
    for call in calls():
        with pytest.raises(ValueError, match="do not fit"):
            call(Shaped(torch.float16, shape, strides), rows, stride)
