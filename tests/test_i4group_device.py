"""Ops of a grouped 4-bit launch, built while one device was current, are refused on another (no GPU needed)."""
from __future__ import annotations

import pytest

import dequantize_mat_vec_amd as dmv
from test_experts_types import DeviceTensor as T


def test_ops_of_another_device():
    import torch
    f32 = torch.float32
    op = (8, 40, T(torch.uint8, 160), T(torch.float16, 16), None, T(f32, 40), T(f32, 8), None)   # 40 columns: refused by the library
    ops = dmv.gemv_i4group_ops([op], 32, 1)
    with pytest.raises(dmv.PestiError):
        dmv.pesti_gemv_group_i4group(ops, 32, 1, stream=0)
    ops.device += 1
    with pytest.raises(ValueError, match="device"):
        dmv.pesti_gemv_group_i4group(ops, 32, 1, stream=0)
    by_hand = (dmv.GemvI4GroupOp * 1)(*ops)
    with pytest.raises(dmv.PestiError):
        dmv.pesti_gemv_group_i4group(by_hand, 32, 1, stream=0)


def test_ops_keep_their_tensors():
    """A tensor that only the call to gemv_i4group_ops named is not freed under the array."""
    import gc
    import weakref

    import torch
    f32 = torch.float32
    x = T(f32, 40)
    gone = weakref.ref(x)
    ops = dmv.gemv_i4group_ops([(8, 40, T(torch.uint8, 160), T(torch.float16, 16), None, x, T(f32, 8), None)], 32, 1)
    del x
    gc.collect()
    assert gone() is not None
    del ops
    gc.collect()
    assert gone() is None
