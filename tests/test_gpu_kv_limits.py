"""The cache, its attention and the 4-bit mat-vecs at the largest counts that the interface names, and two streams at
once."""
from __future__ import annotations

import numpy as np
import pytest

import dequantize_mat_vec_amd as dmv
from gpu_util import announce, guarded_y, guards_intact, to_dev
from kv_reference import Cache, i4_matrix, i4_tolerance, i4_weights
from test_gpu_attention import check, queries, workspace_of
from test_gpu_kv_cache import OnGpu

pytestmark = pytest.mark.gpu


def rng_of(*key):
    return np.random.default_rng([79, *key])


def test_as_many_rows_as_there_may_be():
    announce("attend 4096 rows")
    rng = rng_of(1)
    lengths = rng.integers(0, 4, 4096)
    g = OnGpu(Cache(rng, "f16", 1, 4096, 8, 1, 32, 4096, 1, lengths))
    check(g, queries(rng, 4096, 2, 32), 32 ** -0.5, max_length=8)


@pytest.mark.parametrize("kv,group", [(1, 1024), (1024, 1), (128, 8)])
def test_as_many_heads_as_there_may_be(kv, group):
    announce(f"attend {kv} KV heads, {group} query heads each")
    rng = rng_of(2, kv)
    g = OnGpu(Cache(rng, "i8row", 1, 12, 8, kv, 32, 2, 8, (40, 9)))
    check(g, queries(rng, 2, kv * group, 32), 32 ** -0.5)
    check(g, queries(rng, 2, kv * group, 32), 32 ** -0.5, max_length=64 * 8)


def test_append_of_as_many_rows_as_there_may_be():
    announce("append 2^20 rows")
    import torch
    rows, page, seqs = 1 << 20, 1024, 64
    width = rows // seqs // page
    k, v = (torch.zeros(1, seqs * width, 1, page, 32, dtype=torch.float16, device="cuda") for _ in range(2))
    cache = dmv.kv_cache("f16", 1, seqs * width, page, 1, 32, k, v)
    pages = torch.randperm(seqs * width, device="cuda").to(torch.int32).view(seqs, width)
    lengths = torch.full((seqs,), width * page, dtype=torch.int32, device="cuda")
    table = dmv.kv_table(pages, lengths)
    x = torch.randn(2, rows, 32, device="cuda")
    at = torch.randperm(rows, device="cuda")
    seq, pos = (at // (width * page)).to(torch.int32), (at % (width * page)).to(torch.int32)
    dmv.pesti_cache_append(cache, table, 0, rows, x[0], x[1], seq_ids=seq, positions=pos)
    torch.cuda.synchronize()
    place = pages[seq.long(), pos.long() // page].long() * page + pos.long() % page
    for pool, want in ((k, x[0]), (v, x[1])):
        assert torch.equal(pool.view(-1, 32)[place], want.half())


def test_pages_of_the_largest_pool():
    """2^22 pages, all but the last few held: those are found, and compaction moves them to the holes at the front."""
    announce("extend and compact 2^22 pages")
    import torch
    pages, page, seqs = 1 << 22, 8, 3
    k, v = (torch.zeros(1, pages, 1, page, 32, dtype=torch.int8, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros(1, pages, 1, page, device="cuda") for _ in range(2))
    cache = dmv.kv_cache("i8row", 1, pages, page, 1, 32, k, v, ks, vs)
    refs = torch.ones(pages, dtype=torch.int32, device="cuda")
    refs[-5:] = 0
    refs[1 << 21] = 0
    ids = torch.full((seqs, 4), -1, dtype=torch.int32, device="cuda")
    lengths, status = torch.zeros(seqs, dtype=torch.int32, device="cuda"), torch.full((1,), 9, dtype=torch.int32, device="cuda")
    table = dmv.kv_table(ids, lengths, refs)
    dmv.pesti_cache_extend(cache, table, 3, counts=to_dev(np.array([9, 1, 17], np.int32)), status=status)
    assert status.item() == 0 and ids.tolist() == [[1 << 21, pages - 5, -1, -1], [pages - 4, -1, -1, -1],
                                                   [pages - 3, pages - 2, pages - 1, -1]]
    dmv.pesti_cache_extend(cache, table, 1, counts=to_dev(np.array([8], np.int32)), status=status)
    assert status.item() == 1 and lengths.tolist() == [9, 1, 17]
    k[0, pages - 1, 0, 0] = 7
    refs[1000:1003] = 0
    live = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.empty(dmv.pesti_cache_workspace_bytes(cache, table), dtype=torch.uint8, device="cuda")
    dmv.pesti_cache_compact(cache, table, live, ws)
    torch.cuda.synchronize()
    assert live.item() == pages - 3 and ids[2].tolist() == [1000, 1001, 1002, -1]
    assert ids[0].tolist() == [1 << 21, pages - 5, -1, -1] and (k[0, 1002, 0, 0] == 7).all()
    assert (refs[:pages - 3] == 1).all() and (refs[pages - 3:] == 0).all()


@pytest.mark.parametrize("batch,out,inf", [(2, 3000001, 64), (8, 1000003, 32)])
def test_millions_of_rows(batch, out, inf):
    announce(f"i4group {batch}x{out}x{inf}")
    import torch
    rng = rng_of(3, out)
    m = i4_matrix(rng, out, inf, 32)
    x = rng.standard_normal((batch, inf)).astype(np.float32)
    buf, y = guarded_y(batch * out)
    dmv.pesti_gemv_i4group(out, inf, 32, *(to_dev(v) for v in m), to_dev(x), y, None, batch)
    torch.cuda.synchronize()
    assert guards_intact(buf, batch * out)
    y = y.cpu().numpy().reshape(batch, out).astype(np.float64)
    w = i4_weights(*m, inf, 32)
    exact = x.astype(np.float64) @ w.T
    assert np.all(np.abs(y - exact) <= i4_tolerance(w, x.astype(np.float64)) + 2.0 ** -24 * np.abs(exact))


def test_two_streams_at_once():
    """Attention and 4-bit mat-vecs on two streams side by side, each with its own workspace and outputs."""
    announce("two streams")
    import torch
    rng = rng_of(4)
    g = OnGpu(Cache(rng, "f16", 1, 700, 16, 4, 64, 4, 200, (3000, 40, 1500, 2999)))
    q = [to_dev(queries(rng, 4, 8, 64)).view(4, -1) for _ in range(2)]
    m = [to_dev(v) for v in i4_matrix(rng, 5000, 2048, 64)]
    x = to_dev(rng.standard_normal((6, 2048)).astype(np.float32))

    def work(i, out, stream):
        dmv.pesti_attn_paged(g.cache, g.table, 0, 4, 8, q[i], out[0], 0.125, max_length=3000, workspace=out[2], stream=stream)
        dmv.pesti_gemv_i4group(5000, 2048, 64, *m, x, out[1], None, 6, stream=stream)

    def fresh():
        return torch.full((4, 8, 64), 3.0, device="cuda"), torch.full((6, 5000), 3.0, device="cuda"), workspace_of(g.cache, 4, 8, 3000)

    want = [fresh() for _ in range(2)]
    for i in range(2):
        work(i, want[i], None)
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[fresh() for _ in range(10)] for _ in range(2)]
    torch.cuda.synchronize()
    for n in range(10):
        for i in range(2):
            work(i, got[i][n], streams[i])
    torch.cuda.synchronize()
    for i in range(2):
        for out in got[i]:
            assert torch.equal(out[0], want[i][0]) and torch.equal(out[1], want[i][1])
