"""The calls that the binding makes as a whole in compiled code against the ones that it makes argument by argument
(a stream given): the same bits, the same refusals."""
from __future__ import annotations

import numpy as np
import pytest

import dequantize_mat_vec_amd as dmv
from dequantize_mat_vec_amd import _lib
from gpu_util import announce, to_dev
from kv_reference import Cache, i4_matrix
from test_gpu_attention import queries, workspace_of
from test_gpu_kv_cache import OnGpu

pytestmark = pytest.mark.gpu


def fixture():
    import torch
    dmv.load()
    rng = np.random.default_rng([83, 1])
    g = OnGpu(Cache(rng, "f16", 2, 60, 16, 2, 64, 3, 20, (200, 17, 90)))
    m = [to_dev(v) for v in i4_matrix(rng, 96, 256, 64)]
    u = [to_dev(v) for v in i4_matrix(rng, 96, 256, 64)]
    x, y, bias = to_dev(rng.standard_normal((2, 256)).astype(np.float32)), torch.zeros(2, 96, device="cuda"), torch.ones(96, device="cuda")
    kv = to_dev(rng.standard_normal((3, 2, 128)).astype(np.float32)).view(3, 256)
    q = to_dev(queries(rng, 3, 14, 64)).view(3, -1)
    out = torch.zeros(3, 14, 64, device="cuda")
    ws = workspace_of(g.cache, 3, 14, 320)
    ints = torch.tensor([2, 0, 1], dtype=torch.int32, device="cuda")
    status = torch.full((1,), 5, dtype=torch.int32, device="cuda")
    upkeep = torch.empty(dmv.pesti_cache_workspace_bytes(g.cache, g.table), dtype=torch.uint8, device="cuda")
    return {
        "pesti_cache_extend": (status, dict(cache=g.cache, table=g.table, n=3, seq_ids=ints, counts=ints * 0 - 1, status=status)),
        "pesti_cache_free": (g.arrays["table"], dict(cache=g.cache, table=g.table, n=3, seq_ids=ints - 9)),
        "pesti_cache_fork": (status, dict(cache=g.cache, table=g.table, n=3, parents=ints, children=ints, status=status,
                                          workspace=upkeep)),
        "pesti_cache_compact": (status, dict(cache=g.cache, table=g.table, live=status, workspace=upkeep)),
        "pesti_gemv_i4group": (y, dict(out_features=96, in_features=256, group=64, packed=m[0], scales=m[1], zeros=m[2], x=x, y=y,
                                       bias=bias, batch=2)),
        "pesti_gemv_i4group_swiglu": (y, dict(out_features=96, in_features=256, group=64, gate_packed=m[0], gate_scales=m[1],
                                              gate_zeros=m[2], up_packed=u[0], up_scales=u[1], up_zeros=None, x=x, h=y, batch=2)),
        "pesti_cache_append": (g.arrays["k"], dict(cache=g.cache, table=g.table, layer=1, rows=3, k=kv, v=kv[:, 128:], stride=256,
                                                   seq_ids=ints, positions=ints)),
        "pesti_attn_paged": (out, dict(cache=g.cache, table=g.table, layer=1, rows=3, heads=14, q=q, y=out, scale=0.125,
                                       max_length=320, seq_ids=ints, workspace=ws)),
    }


NAMES = ["pesti_gemv_i4group", "pesti_gemv_i4group_swiglu", "pesti_cache_append", "pesti_attn_paged"]
# (as the fixture has them these change nothing: no more tokens, no such sequence, children that are not empty; and pages
# that lie in front already once they have been moved there)
UPKEEP = ["pesti_cache_extend", "pesti_cache_free", "pesti_cache_fork", "pesti_cache_compact"]


@pytest.mark.parametrize("name", NAMES)
def test_made_and_the_same(name, monkeypatch):
    announce(f"fast {name}")
    import torch
    result, args = fixture()[name]
    made = []
    fast = "_call_" + name[len("pesti_"):]
    inner = getattr(_lib, fast)

    def watch(*args):
        made.append(inner(*args))
        return made[-1]
    monkeypatch.setattr(_lib, fast, watch)
    outs = []
    for stream in (None, torch.cuda.current_stream()):
        result.zero_()
        assert getattr(dmv, name)(**args, stream=stream) == 0
        outs.append(result.clone())
    assert made == [0] and torch.equal(*outs) and outs[0].any()
    side = torch.cuda.Stream()
    result.zero_()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):   # the current stream
        assert getattr(dmv, name)(**args) == 0
    side.synchronize()
    assert made == [0, 0] and torch.equal(result, outs[0])


def bad(value):
    """What may be wrong with an argument, by its kind."""
    import torch
    if isinstance(value, torch.Tensor):
        yield "on the host", value.cpu()
        yield "of another type", value.to(torch.bfloat16 if value.is_floating_point() else torch.int64)
        if value.dim() > 1:
            yield "not contiguous", torch.cat([value, value], -1)[:, ::2] if value.dim() == 2 else value.transpose(0, 1)
        yield "too small", value.reshape(-1)[:1]
        yield "no tensor", "pool"
    elif isinstance(value, int):
        yield "negative", -3
        yield "too large", 1 << 40
        yield "no number", "5"


@pytest.mark.parametrize("name", UPKEEP)
def test_upkeep_is_made(name, monkeypatch):
    announce(f"fast {name}")
    import torch
    _, args = fixture()[name]
    made = []
    fast = "_call_" + name[len("pesti_"):]
    inner = getattr(_lib, fast)
    monkeypatch.setattr(_lib, fast, lambda *a: made.append(inner(*a)) or made[-1])
    arrays = [t for t in (*args["table"].tensors, *args["cache"].tensors, args.get("status", args.get("live"))) if t is not None]
    after = []
    for stream in (None, torch.cuda.current_stream()):
        assert getattr(dmv, name)(**args, stream=stream) == 0
        after.append([t.clone() for t in arrays])
    assert made == [0] and all(torch.equal(a, b) for a, b in zip(*after))


@pytest.mark.parametrize("name", NAMES + UPKEEP)
def test_the_same_refusals(name):
    announce(f"fast {name} refusals")
    import torch
    _, args = fixture()[name]
    stream = torch.cuda.current_stream()
    seen = 0
    for key, value in args.items():
        for what, wrong in bad(value):
            if key in ("rows", "batch", "stride", "max_length", "n") and what == "too large":
                continue   # sizes of memory that no test has
            answers = []
            for given in (None, stream):
                try:
                    answers.append(("status", getattr(dmv, name)(**{**args, key: wrong}, stream=given)))
                except Exception as e:
                    answers.append((type(e), str(e)))
            assert answers[0] == answers[1], (key, what)
            seen += answers[0][0] != "status"
    assert seen >= (6 if name in UPKEEP else 20)
    torch.cuda.synchronize()


def test_other_structs_are_looked_at():
    """A table with too few counts, a struct filled in by hand."""
    announce("fast structs")
    import torch
    out, args = fixture()["pesti_attn_paged"]
    table = args["table"]
    short = dmv.kv_table(table.tensors[0], table.tensors[1], torch.zeros(5, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError, match="refs holds 5"):
        dmv.pesti_attn_paged(**{**args, "table": short})
    by_hand = dmv.KvTable(table.seqs, table.width, table.table, table.lengths, None)
    out.zero_()
    assert dmv.pesti_attn_paged(**{**args, "table": by_hand}) == 0
    got = out.clone()
    assert dmv.pesti_attn_paged(**args) == 0 and torch.equal(got, out)
