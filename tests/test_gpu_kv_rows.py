"""Rows that a tensor does not have, though its memory goes on behind them: refused by the calls made as a whole too."""
from __future__ import annotations

import pytest

import dequantize_mat_vec_amd as dmv
from gpu_util import announce
from test_gpu_fast_calls import fixture

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("given", [False, True])
def test_rows_that_are_not_there(given):
    announce(f"rows that are not there, stream given {given}")
    import torch
    cases = fixture()
    stream = torch.cuda.current_stream() if given else None
    out, attend = cases["pesti_attn_paged"]
    pool, append = cases["pesti_cache_append"]
    q, k = attend["q"], append["k"]
    wide = torch.cat([q, q], 1)
    for bad in (dict(q=q[:2]), dict(q=q[:, :448]), dict(q=wide[:, :448], q_stride=wide.shape[1]), dict(q=q.reshape(-1)[:-1], q_stride=896)):
        with pytest.raises(ValueError, match="do not fit"):
            dmv.pesti_attn_paged(**{**attend, **bad}, stream=stream)
    for bad in (dict(k=k[:2]), dict(v=k[:2, 128:]), dict(k=k[:, :64]), dict(v=k[:, 192:])):
        with pytest.raises(ValueError, match="do not fit"):
            dmv.pesti_cache_append(**{**append, **bad}, stream=stream)
    assert dmv.pesti_attn_paged(**{**attend, "q": wide[:, :896]}, stream=stream) == 0
    got = out.clone()
    assert dmv.pesti_attn_paged(**attend, stream=stream) == 0 and torch.equal(out, got)
    assert dmv.pesti_cache_append(**{**append, "k": k[:, :128]}, stream=stream) == 0
    torch.cuda.synchronize()
