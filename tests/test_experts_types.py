"""Element types of the tensors that the 8-bit and expert calls take, checked
by the binding before the library is called (safe without a GPU: every call
here has an in_features that the library refuses, so nothing is launched)."""
from __future__ import annotations

import pytest

import dequantize_mat_vec_amd as dmv
from dequantize_mat_vec_amd import _lib

K = 40   # not a multiple of 32: refused by the library


class DeviceTensor:
    """What the binding asks of a tensor on device 0; its address is never read."""

    def __init__(self, dtype, count):
        self.dtype, self.nbytes = dtype, count * dtype.itemsize

    def get_device(self):
        return 0

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 0x100000


def calls(torch):
    """Every call with tensors of the types that it asks for, by name: (function, positional arguments, keywords);
    and for each tensor the types that hold as many bytes or more and are not it."""
    f32, f16, i8, i32 = torch.float32, torch.float16, torch.int8, torch.int32
    t = DeviceTensor
    m, n, e = 4, 8, 2
    not_f16, not_f32, not_i8 = (torch.bfloat16, f32, torch.int16), (torch.int32, torch.float64), (torch.uint8, f16)

    def experts(form, y):
        v = f16 if form == "f16" else i8
        kw = {} if form == "f16" else dict(w_scales=t(f32, e * n), x_scales=t(f32, m))
        return ("pesti_gemm_experts", dict(fmt=form, rows=m, experts=e, out_features=n, in_features=K, offsets=t(i32, e + 1),
                                           w=t(v, e * n * K), x_tokens=m, x=t(v, m * K), y=t(y, m * n), y_format="f16" if y == f16 else "f32", **kw),
                dict(w=not_f16 if v == f16 else not_i8, x=not_f16 if v == f16 else not_i8, y=not_f16 if y == f16 else not_f32))

    def swiglu(form, h):
        v = f16 if form == "f16" else i8
        kw = {} if form == "f16" else dict(gate_scales=t(f32, e * n), up_scales=t(f32, e * n), x_scales=t(f32, m))
        bad = not_f16 if v == f16 else not_i8
        return ("pesti_gemm_experts_swiglu", dict(fmt=form, rows=m, experts=e, out_features=n, in_features=K, offsets=t(i32, e + 1),
                                                  w_gate=t(v, e * n * K), w_up=t(v, e * n * K), x_tokens=m, x=t(v, m * K), h=t(h, m * n),
                                                  h_format="f16" if h == f16 else "f32", **kw),
                dict(w_gate=bad, w_up=bad, x=bad, h=not_f16 if h == f16 else not_f32))

    def quant(x):
        return ("pesti_quant_i8token", dict(x_format="f16" if x == f16 else "f32", m=m, in_features=K, x=t(x, m * K), codes=t(i8, m * K),
                                            scales=t(f32, m)),
                dict(x=not_f16 if x == f16 else not_f32, codes=not_i8))

    def product(y):
        return ("pesti_gemm_i8row_i8token", dict(m=m, out_features=n, in_features=K, codes=t(i8, n * K), row_scales=t(f32, n),
                                                 x_codes=t(i8, m * K), x_scales=t(f32, m), y=t(y, m * n), y_format="f16" if y == f16 else "f32"),
                dict(codes=not_i8, x_codes=not_i8, y=not_f16 if y == f16 else not_f32))

    return [quant(f16), quant(f32), product(f16), product(f32), experts("f16", f32), experts("f16", f16), experts("i8row", f32),
            swiglu("f16", f16), swiglu("i8row", f32)]


def test_tensors_of_the_types_asked_for_reach_the_library():
    import torch
    for name, kw, _ in calls(torch):
        with pytest.raises(_lib.PestiError) as e:
            getattr(dmv, name)(**kw, stream=0)
        assert e.value.status == _lib.PESTI_ERR_SHAPE, name


def test_tensors_of_other_types_are_refused():
    """bfloat16 has binary16's size, and more bytes than needed pass a check of sizes: each was read as the type
    that the call takes."""
    import torch
    for name, kw, others in calls(torch):
        for what, types in others.items():
            for dtype in types:
                bad = dict(kw, **{what: DeviceTensor(dtype, kw[what].nbytes // kw[what].dtype.itemsize)})
                with pytest.raises(ValueError, match=rf"^{what} must be a "):
                    getattr(dmv, name)(**bad, stream=0)


def test_binary16_may_be_held_as_its_bits():
    """uint16 tensors, the type of binary16 in the C ABI, as the small-M GEMMs are given them."""
    import torch
    for name, kw, others in calls(torch):
        for what in others:
            if kw[what].dtype == torch.float16:
                bits = dict(kw, **{what: DeviceTensor(torch.uint16, kw[what].nbytes // 2)})
                with pytest.raises(_lib.PestiError) as e:
                    getattr(dmv, name)(**bits, stream=0)
                assert e.value.status == _lib.PESTI_ERR_SHAPE, (name, what)


def test_a_tensor_too_small_is_named_by_its_size():
    import torch
    for name, kw, others in calls(torch):
        for what in others:
            bad = dict(kw, **{what: DeviceTensor(kw[what].dtype, kw[what].nbytes // kw[what].dtype.itemsize - 1)})
            with pytest.raises(ValueError, match=rf"^{what} holds "):
                getattr(dmv, name)(**bad, stream=0)


def test_addresses_have_no_type():
    """Raw device addresses pass as they are, with the format that the caller gives."""
    import torch
    for name, kw, others in calls(torch):
        raw = {k: 0x100000 if isinstance(v, DeviceTensor) else v for k, v in kw.items()}
        with pytest.raises(_lib.PestiError) as e:
            getattr(dmv, name)(**raw, stream=0)
        assert e.value.status == _lib.PESTI_ERR_SHAPE, name
