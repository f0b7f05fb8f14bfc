"""Tensors without strides or memory of their own (sparse ones, those of a torch.vmap) are refused with an error
(torch's own, or the binding's), by every call and for each of its tensors; the process goes on."""
from __future__ import annotations

import numpy as np
import pytest

import dequantize_mat_vec_amd as dmv
from gpu_util import announce, to_dev
from test_gpu_fast_calls import NAMES, UPKEEP, fixture

pytestmark = pytest.mark.gpu


def refused(call, kind, value):
    """The error of call(a tensor of that layout)."""
    import torch
    flat = value if value.dim() == 2 else value.reshape(1, -1)
    with pytest.raises((RuntimeError, ValueError)) as e:
        if kind == "vmap":
            torch.vmap(lambda t: (call(t), t)[1])(torch.stack([value, value]))
        else:
            call(flat.to_sparse() if kind == "sparse" else flat.to_sparse_csr())
    assert not isinstance(e.value, dmv.PestiError), e.value
    return str(e.value)


@pytest.mark.parametrize("kind", ["sparse", "csr", "vmap"])
@pytest.mark.parametrize("name", NAMES + UPKEEP)
def test_layouts_of_the_calls_made_as_a_whole(name, kind):
    announce(f"layout {name} {kind}")
    import torch
    _, args = fixture()[name]
    seen = 0
    for key, value in args.items():
        if not isinstance(value, torch.Tensor):
            continue
        texts = {refused(lambda t, s=stream: getattr(dmv, name)(**{**args, key: t}, stream=s), kind, value).splitlines()[0]
                 for stream in (None, torch.cuda.current_stream())}
        assert len(texts) == 1, (key, texts)
        seen += 1
    assert seen >= 1
    torch.cuda.synchronize()


@pytest.mark.parametrize("kind", ["sparse", "csr", "vmap"])
def test_layouts_of_calls_checked_argument_by_argument(kind):
    announce(f"layout 8-bit and expert calls {kind}")
    import torch
    x = to_dev(np.ones((3, 64), np.float32))
    codes, scales = torch.empty(3, 64, dtype=torch.int8, device="cuda"), torch.empty(3, device="cuda")
    assert dmv.pesti_quant_i8token("f32", 3, 64, x, codes, scales) == 0
    for call, value in ((lambda t: dmv.pesti_quant_i8token("f32", 3, 64, t, codes, scales), x),
                        (lambda t: dmv.pesti_quant_i8token("f32", 3, 64, x, codes, t), scales),
                        (lambda t: dmv.pesti_dequant_i4group(1, 64, 32, t, scales, None, x), codes.to(torch.uint8)),
                        (lambda t: dmv.kv_table(t, torch.zeros(3, dtype=torch.int32, device="cuda")), codes.to(torch.int32))):
        refused(call, kind, value)
    torch.cuda.synchronize()
