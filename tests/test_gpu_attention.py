"""Attention of one new token over the paged cache on the GPU against the 64-bit
form: head layouts, dimensions, page sizes and lengths that end anywhere, splits
of the length, rows without tokens, pages that are not there, values in places
that must not be read, offsets past 32 bits, streams and graphs."""
from __future__ import annotations

import numpy as np
import pytest

import dequantize_mat_vec_amd as dmv
from gpu_util import CANARY_BITS, GUARD, announce, guarded_y, guards_intact, to_dev
from kv_reference import Cache
from test_gpu_kv_cache import OnGpu, ints

pytestmark = pytest.mark.gpu


def rng_of(*key):
    return np.random.default_rng([73, *key])


def workspace_of(cache, rows, heads, max_length):
    import torch
    n = dmv.pesti_attn_paged_workspace_bytes(cache, rows, heads, max_length)
    assert n >= 0
    return torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda") if n else None   # NaN in every float


def attend(g, layer, q, scale, seq_ids=None, y_kind=np.float32, max_length=None, q_pad=0):
    """y float64 [rows][heads][d] of the library, guards checked."""
    import torch
    rows, heads, d = q.shape
    if max_length is None:
        max_length = max(1, int(g.c.lengths.max(initial=1)))
    wide = np.full((rows, heads * d + q_pad), np.nan, q.dtype)
    wide[:, :heads * d] = q.reshape(rows, -1)
    n = q.size
    if y_kind == np.float32:
        buf, y = guarded_y(n)
    else:
        buf = torch.full((GUARD + n + GUARD,), CANARY_BITS & 0x7FFF, dtype=torch.int16, device="cuda").view(torch.float16)
        y = buf[GUARD:GUARD + n]
    dmv.pesti_attn_paged(g.cache, g.table, layer, rows, heads, to_dev(wide), y, scale, max_length=max_length,
                         seq_ids=None if seq_ids is None else to_dev(np.asarray(seq_ids, np.int32)),
                         workspace=workspace_of(g.cache, rows, heads, max_length))
    torch.cuda.synchronize()
    if y_kind == np.float32:
        assert guards_intact(buf, n)
    else:
        bits = buf.view(torch.int16).cpu().numpy()
        assert (bits[:GUARD] == CANARY_BITS & 0x7FFF).all() and (bits[GUARD + n:] == CANARY_BITS & 0x7FFF).all()
    return y.cpu().numpy().reshape(q.shape).astype(np.float64)


def check(g, q, scale, layer=0, seq_ids=None, y_kind=np.float32, max_length=None, q_pad=0):
    y = attend(g, layer, q, scale, seq_ids, y_kind, max_length, q_pad)
    exact, bound = g.c.attend(layer, q, scale, seq_ids)
    half = 2.0 ** -24 if y_kind == np.float32 else 2.0 ** -11
    tiny = 0.0 if y_kind == np.float32 else 2.0 ** -25
    tol = bound + half * (np.abs(exact) + bound) + tiny
    err = np.abs(y - exact)
    assert np.all(err <= tol), (float((err / np.maximum(tol, 1e-300)).max()), np.unravel_index(np.argmax(err - tol), err.shape))


def queries(rng, rows, heads, d, kind=np.float32, size=1.0):
    return (rng.standard_normal((rows, heads, d)) * size).astype(kind)


# every head dimension, query heads per KV head around the tile's width, page sizes on both sides of the token tile
LAYOUTS = [(32, 1, 1, 8), (32, 2, 7, 16), (64, 2, 7, 16), (64, 12, 1, 64), (96, 1, 3, 8), (96, 2, 8, 32), (128, 2, 4, 16),
           (128, 1, 9, 128), (160, 1, 5, 8), (160, 2, 2, 64), (192, 1, 16, 32), (224, 1, 6, 16), (224, 2, 1, 256), (256, 1, 8, 8),
           (256, 1, 4, 64), (64, 1, 17, 16), (128, 1, 40, 32), (64, 1, 71, 8)]


@pytest.mark.parametrize("d,kv,group,page", LAYOUTS)
@pytest.mark.parametrize("fmt", ["f16", "i8row"])
def test_layouts(d, kv, group, page, fmt):
    announce(f"attend d {d} kv {kv} group {group} page {page} {fmt}")
    rng = rng_of(1, d, group, page)
    lengths = [1, page - 1, page, page + 1, 31, 32, 33, 64, 65, 200, 0]
    width = -(-200 // page) + 1
    pages = sum(-(-n // page) for n in lengths) + 2
    g = OnGpu(Cache(rng, fmt, 2, pages, page, kv, d, len(lengths), max(width, 2), lengths))
    check(g, queries(rng, len(lengths), kv * group, d), d ** -0.5, layer=1)


@pytest.mark.parametrize("q_kind,y_kind", [(np.float32, np.float16), (np.float16, np.float32), (np.float16, np.float16)])
@pytest.mark.parametrize("d,kv,group,page", [(64, 2, 7, 16), (128, 2, 12, 32), (96, 1, 1, 8)])
def test_types(q_kind, y_kind, d, kv, group, page):
    announce(f"attend {q_kind.__name__} -> {y_kind.__name__} d {d}")
    rng = rng_of(2, d)
    g = OnGpu(Cache(rng, "f16", 1, 40, page, kv, d, 4, 16, [5, 70, 128, 33]))
    check(g, queries(rng, 4, kv * group, d, q_kind), d ** -0.5, y_kind=y_kind, q_pad=16)


@pytest.mark.parametrize("length", [1, 2, 16, 17, 127, 128, 129, 255, 256, 257, 511, 513, 1023, 1025, 2047, 4097])
@pytest.mark.parametrize("fmt,page", [("f16", 16), ("i8row", 32), ("f16", 256)])
def test_one_row_of_every_length(length, fmt, page):
    announce(f"attend length {length} {fmt} page {page}")
    rng = rng_of(3, length, page)
    g = OnGpu(Cache(rng, fmt, 1, -(-length // page) + 1, page, 2, 64, 1, -(-length // page), [length]))
    check(g, queries(rng, 1, 14, 64, size=3.0), 0.125)


@pytest.mark.parametrize("max_length", [1, 100, 5000, 1 << 20, 1 << 30])
def test_any_bound_of_the_length_gives_the_result(max_length):
    """The bound chooses the split only: one that is far too small or large changes no result."""
    announce(f"attend max_length {max_length}")
    rng = rng_of(4)
    g = OnGpu(Cache(rng, "f16", 1, 120, 32, 1, 64, 3, 100, [3001, 40, 0]))
    check(g, queries(rng, 3, 4, 64), 0.125, max_length=max_length)


@pytest.mark.parametrize("fmt", ["f16", "i8row"])
def test_long(fmt):
    announce(f"attend long {fmt}")
    rng = rng_of(5)
    g = OnGpu(Cache(rng, fmt, 1, 1400, 64, 2, 64, 2, 1100, [70001, 17000]))
    check(g, queries(rng, 2, 8, 64, size=2.0), 0.125)


def test_peaked_scores():
    """Scores of hundreds: the running maximum rises token by token, or the first token outweighs all others."""
    announce("attend peaked scores")
    rng = rng_of(6)
    c = Cache(rng, "f16", 1, 20, 32, 1, 64, 2, 10, [300, 300])
    q = np.zeros((2, 2, 64), np.float32)
    q[:, :, 0] = 1.0
    for s, order in ((0, np.arange(300)), (1, np.arange(300)[::-1])):
        for t in range(300):
            c.k[0, c.table[s, t // 32], 0, t % 32, 0] = order[t]
    check(OnGpu(c), q, 1.0)
    check(OnGpu(c), -q, 1.0)


def test_magnitudes():
    announce("attend magnitudes")
    rng = rng_of(7)
    for spread, size, scale in ((1e-3, 1e-20, 1e21), (200.0, 1e-4, 1.0), (1.0, 1e30, 1e-31), (1.0, 1e-38, 1e37), (1.0, 1.0, 0.0),
                                (1.0, 1.0, -0.3)):
        g = OnGpu(Cache(rng, "f16", 1, 12, 16, 2, 96, 2, 6, [90, 7], spread=spread))
        check(g, queries(rng, 2, 6, 96, size=size), scale)


def test_rows_of_any_sequence():
    """Rows name sequences in any order, twice, or none at all."""
    announce("attend rows")
    rng = rng_of(8)
    c = Cache(rng, "f16", 1, 60, 16, 2, 64, 6, 9, [100, 0, 33, 140, 16, 5])
    c.lengths[5] = -7
    g = OnGpu(c)
    seq_ids = [3, 1, 0, 3, -1, 6, 2, 5, 4, 0, 2147483647]
    q = queries(rng, len(seq_ids), 6, 64)
    check(g, q, 0.125, seq_ids=seq_ids)
    y = attend(g, 0, q, 0.125, seq_ids)
    for r in (1, 4, 5, 7, 10):
        assert not y[r].any()


def test_lengths_past_the_table():
    announce("attend a length past the table")
    rng = rng_of(9)
    c = Cache(rng, "f16", 1, 12, 16, 1, 64, 2, 4, [64, 64])
    c.lengths[:] = 65, 2147483647
    check(OnGpu(c), queries(rng, 2, 3, 64), 0.125, max_length=64)


@pytest.mark.parametrize("page", [8, 16, 64])
def test_pages_that_are_not_there_are_left_out(page):
    announce(f"attend bad pages, page {page}")
    rng = rng_of(10, page)
    n = 6 * page + 3
    c = Cache(rng, "f16", 1, 40, page, 2, 64, 4, 7, [n, n, n, page])
    c.table[0, [0, 3]] = -1, 40
    c.table[1, 6] = 2147483647
    c.table[2, :] = -2147483648
    c.table[3, 0] = 1 << 20
    g = OnGpu(c)
    q = queries(rng, 4, 4, 64)
    check(g, q, 0.125)
    y = attend(g, 0, q, 0.125)
    assert not y[2:].any()


@pytest.mark.parametrize("fmt", ["f16", "i8row"])
@pytest.mark.parametrize("page", [8, 32, 128])
def test_places_behind_the_last_token_are_not_read_into_the_result(fmt, page):
    announce(f"attend junk behind the end {fmt} page {page}")
    rng = rng_of(11, page)
    lengths = [1, 7, 30, 33, 100, 128]
    c = Cache(rng, fmt, 1, 60, page, 2, 64, 6, 20, lengths)
    taken = np.zeros((c.pages, page), bool)
    for s, n in enumerate(lengths):
        for t in range(n):
            taken[c.table[s, t // page], t % page] = True
    for name in ("k", "v"):
        x = getattr(c, name).transpose(1, 3, 0, 2, 4)   # [pages][page] first
        if fmt == "f16":
            x[~taken] = np.where(rng.random(x[~taken].shape) < 0.5, np.nan, np.inf)
        else:
            x[~taken] = -128
            getattr(c, name + "_scales").transpose(1, 3, 0, 2)[~taken] = np.where(rng.random() < 0.5, np.nan, -np.inf)
    c.table[:, -1] = 2147483647   # entries behind a sequence's pages are not read
    check(OnGpu(c), queries(rng, 6, 14, 64), 0.125)


def test_not_finite():
    """A NaN or infinity stays in the heads, and of V in the values, that it enters."""
    announce("attend infinities and NaN")
    rng = rng_of(12)
    c = Cache(rng, "f16", 1, 40, 16, 2, 64, 5, 8, [50, 50, 50, 50, 50])
    c.k[0, c.table[1, 2], 0, 3, 9] = np.nan     # KV head 0 of sequence 1
    c.v[0, c.table[2, 1], 1, 4, 20] = np.inf    # one value of KV head 1 of sequence 2
    q = queries(rng, 5, 6, 64)
    q[3, 2, 5] = np.nan
    c.k[0, c.table[4, 0], 1, 0] = 0
    c.k[0, c.table[4, 0], 1, 0, 7] = -np.inf    # a token of weight zero where q is positive
    q[4, 3:, 7] = np.abs(q[4, 3:, 7]) + 0.1
    g = OnGpu(c)
    y = attend(g, 0, q, 0.125)
    with np.errstate(invalid="ignore"):
        exact, bound = c.attend(0, q, 0.125)
    tol = np.nan_to_num(bound, nan=1.0, posinf=1.0) + 2.0 ** -24 * np.abs(exact)
    ok = np.isfinite(exact)
    assert np.isnan(y[1, :3]).all() and np.isfinite(y[1, 3:]).all()
    assert np.all(y[2, 3:, 20] == np.inf)
    assert np.isnan(y[3, 2]).all() and np.isfinite(y[3, [0, 1, 3, 4, 5]]).all()
    assert np.isfinite(y[2][:, np.arange(64) != 20]).all() and np.isfinite(y[4]).all()
    assert np.all(np.abs(y[0] - exact[0]) <= tol[0])
    k, there = c.rows("k", 0, 4, 1)
    v, _ = c.rows("v", 0, 4, 1)
    for h in (3, 4, 5):
        s = k[1:] @ q[4, h].astype(np.float64) * 0.125
        p = np.exp(s - s.max())
        assert np.all(np.abs(y[4, h] - p @ v[1:] / p.sum()) <= 1e-4)
    assert ok[0].all()


def test_every_score_minus_infinity_is_a_row_of_zeros():
    announce("attend all scores -inf")
    rng = rng_of(13)
    c = Cache(rng, "f16", 1, 4, 16, 1, 64, 1, 2, [20])
    c.k[:] = 1.0
    c.k[..., 3] = -np.inf
    y = attend(OnGpu(c), 0, np.ones((1, 2, 64), np.float32), 1.0)
    assert not y.any()


def test_offsets_past_32_bits():
    """Pages whose bytes lie past 4 GiB of K and of V."""
    announce("attend past 4 GiB")
    import torch
    pages, page, kv, d = 36000, 64, 8, 128   # 4.7 GB each
    rng = rng_of(14)
    k, v = (torch.zeros(1, pages, kv, page, d, dtype=torch.float16, device="cuda") for _ in range(2))
    used = np.array([35999, 0, 32768, 33001, 35000, 16384], np.int32)
    c = Cache(rng, "f16", 1, 6, page, kv, d, 2, 4, [200, 100], shuffle=False)
    for x, host in ((k, c.k), (v, c.v)):
        x[0, torch.from_numpy(used.astype(np.int64)).cuda()] = to_dev(host[0])
    big = c.table.copy()
    big[big >= 0] = used[big[big >= 0]]
    cache = dmv.kv_cache("f16", 1, pages, page, kv, d, k, v)
    lengths = to_dev(c.lengths)
    table = dmv.kv_table(to_dev(big), lengths, torch.ones(pages, dtype=torch.int32, device="cuda"))
    q = queries(rng, 2, 16, d)
    y = torch.empty(2, 16, d, device="cuda")
    dmv.pesti_attn_paged(cache, table, 0, 2, 16, to_dev(q).view(2, -1), y, d ** -0.5, max_length=200,
                         workspace=workspace_of(cache, 2, 16, 200))
    exact, bound = c.attend(0, q, d ** -0.5)
    assert np.all(np.abs(y.cpu().numpy() - exact) <= bound + 2.0 ** -24 * np.abs(exact))
    # rows written there too
    x = rng.standard_normal((2, 2, kv * d)).astype(np.float16)
    dmv.pesti_cache_append(cache, table, 0, 2, to_dev(x[0]), to_dev(x[1]))
    torch.cuda.synchronize()
    for r, n in enumerate((200, 100)):
        p = big[r, (n - 1) // page]
        assert np.array_equal(k[0, int(p), :, (n - 1) % page].cpu().numpy().reshape(-1), x[0, r])
        assert np.array_equal(v[0, int(p), :, (n - 1) % page].cpu().numpy().reshape(-1), x[1, r])
    src = torch.tensor([35999], dtype=torch.int32, device="cuda")
    dmv.pesti_cache_copy_pages(cache, 1, src, torch.tensor([34567], dtype=torch.int32, device="cuda"))
    assert torch.equal(k[0, 34567], k[0, 35999]) and torch.equal(v[0, 34567], v[0, 35999])


def test_same_bits_every_time_and_on_another_stream():
    announce("attend repeated")
    import torch
    rng = rng_of(15)
    g = OnGpu(Cache(rng, "i8row", 1, 400, 16, 2, 128, 3, 300, [4000, 1500, 3]))
    q, first = to_dev(queries(rng, 3, 8, 128)).view(3, -1), None
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for i in range(6):
        y, ws = torch.full((3, 8, 128), 5.0, device="cuda"), workspace_of(g.cache, 3, 8, 4000)
        torch.cuda.synchronize()
        dmv.pesti_attn_paged(g.cache, g.table, 0, 3, 8, q, y, 0.1, max_length=4000, workspace=ws, stream=side if i % 2 else None)
        torch.cuda.synchronize()
        first = y if first is None else first
        assert torch.equal(y, first)


def test_two_graphs_share_a_workspace():
    """Two captured calls over one workspace, replayed in turn with eager work between, lengths growing."""
    announce("attend captured")
    import torch
    rng = rng_of(16)
    c = Cache(rng, "f16", 2, 300, 16, 2, 64, 2, 140, [900, 2000])
    g = OnGpu(c)
    q, y = to_dev(queries(rng, 2, 14, 64)).view(2, -1), [torch.empty(2, 14, 64, device="cuda") for _ in range(2)]
    ws = workspace_of(g.cache, 2, 14, 2100)

    def call(layer, out):
        dmv.pesti_attn_paged(g.cache, g.table, layer, 2, 14, q, out, 0.125, max_length=2100, workspace=ws)

    torch.cuda.synchronize()
    graphs = []
    for layer in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            call(layer, y[layer])
    for i in range(5):
        for layer in (i % 2, 1 - i % 2):
            y[layer].fill_(3.0)
            graphs[layer].replay()
            torch.cuda.synchronize()
            want = torch.empty(2, 14, 64, device="cuda")
            call(layer, want)
            torch.cuda.synchronize()
            assert torch.equal(y[layer], want), (i, layer)
            exact, bound = c.attend(layer, q.cpu().numpy().reshape(2, 14, 64), 0.125)
            assert np.all(np.abs(want.cpu().numpy() - exact) <= bound + 2.0 ** -24 * np.abs(exact))
        dmv.pesti_cache_extend(g.cache, g.table, 2, None, ints(7, 13), g.status)
        assert c.extend([0, 1], [7, 13]) == 0 == int(g.status[0])
        q.copy_(to_dev(queries(rng, 2, 14, 64)).view(2, -1))


def test_a_decode_step():
    """The calls of one layer's step in a row, captured: 4-bit Q/K/V projections, pages, cache rows, attention, O projection
    and the feed-forward input, against the same steps in 64 bits."""
    announce("decode step")
    import torch
    from kv_reference import i4_matrix, i4_weights, silu
    rng = rng_of(17)
    hidden, heads, kv, d, ffn, batch, group = 224, 7, 1, 32, 96, 3, 32
    c = Cache(rng, "f16", 1, 40, 8, kv, d, batch, 12, [21, 7, 40])
    g = OnGpu(c)
    shapes = dict(q=(heads * d, hidden), k=(kv * d, hidden), v=(kv * d, hidden), o=(hidden, heads * d), gate=(ffn, hidden), up=(ffn, hidden))
    host = {n: i4_matrix(rng, *s, group, scale=0.02) for n, s in shapes.items()}
    dev = {n: tuple(to_dev(a) for a in m) for n, m in host.items()}
    w = {n: i4_weights(*m, shapes[n][1], group) for n, m in host.items()}
    x = to_dev(rng.standard_normal((batch, hidden)).astype(np.float32))
    q, k, v, y, o, h = (torch.empty(batch, n, device="cuda") for n in (heads * d, kv * d, kv * d, heads * d, hidden, ffn))
    ws = workspace_of(g.cache, batch, heads, 96)
    ops = dmv.gemv_i4group_ops([(*shapes[n], *dev[n], x, out, None) for n, out in (("q", q), ("k", k), ("v", v))], group, batch)

    def step():
        dmv.pesti_gemv_group_i4group(ops, group, batch)
        dmv.pesti_cache_extend(g.cache, g.table, batch, None, None, g.status)
        dmv.pesti_cache_append(g.cache, g.table, 0, batch, k, v)
        dmv.pesti_attn_paged(g.cache, g.table, 0, batch, heads, q, y, d ** -0.5, max_length=96, workspace=ws)
        dmv.pesti_gemv_i4group(hidden, heads * d, group, *dev["o"], y, o, None, batch)
        dmv.pesti_gemv_i4group_swiglu(ffn, hidden, group, *dev["gate"], *dev["up"], o, h, batch)

    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(6):
        new = rng.standard_normal((batch, hidden)).astype(np.float32)
        x.copy_(to_dev(new))
        graph.replay()
        torch.cuda.synchronize()
        xd = new.astype(np.float64)
        assert c.extend(range(batch), [1] * batch) == 0 == int(g.status[0])
        # K and V are rounded to binary16: from the library's own float32 values, which are checked apart
        for name, t in (("q", q), ("k", k), ("v", v)):
            assert np.allclose(t.cpu().numpy(), xd @ w[name].T, rtol=0, atol=1e-4)
        c.append(0, k.cpu().numpy().reshape(batch, kv, d), v.cpu().numpy().reshape(batch, kv, d), range(batch), c.lengths - 1)
        g.same()
        ya, bound = c.attend(0, q.cpu().numpy().reshape(batch, heads, d), d ** -0.5)
        got = y.cpu().numpy().reshape(batch, heads, d)
        assert np.all(np.abs(got - ya) <= bound + 2.0 ** -24 * np.abs(ya))
        oa = y.cpu().numpy().astype(np.float64) @ w["o"].T
        assert np.allclose(o.cpu().numpy(), oa, rtol=0, atol=1e-4)
        ha = o.cpu().numpy().astype(np.float64)
        assert np.allclose(h.cpu().numpy(), silu(ha @ w["gate"].T) * (ha @ w["up"].T), rtol=1e-4, atol=1e-4)


# how a sequence is cut and its parts are joined: one part of eight wavefronts, up to 8 parts by threads, more by
# workgroups of 128, 64 or 32 dimensions; parts of 4 tiles and of 8; rows that lack most of the parts
CUTS = [(32, 1, 3, 16, 200), (64, 2, 7, 16, 1000), (64, 8, 2, 32, 5000), (128, 8, 4, 64, 900), (128, 4, 2, 64, 9000), (96, 1, 4, 32, 3000),
        (256, 1, 8, 64, 6000), (160, 2, 3, 128, 40000), (32, 1, 20, 64, 60000), (192, 12, 1, 16, 1100)]


@pytest.mark.parametrize("d,kv,group,page,longest", CUTS)
@pytest.mark.parametrize("rows", [1, 5, 40])
def test_cuts(d, kv, group, page, longest, rows):
    announce(f"attend cut d {d} kv {kv} group {group} page {page} longest {longest} rows {rows}")
    rng = rng_of(17, d, longest, rows)
    longest = longest // (1 if rows == 1 else (3 if rows == 5 else 20))
    lengths = [longest] + [int(n) for n in rng.integers(0, longest // 2 + 1, rows - 1)]
    if rows > 2:
        lengths[1:3] = [0, 1]
    width = -(-longest // page)
    c = Cache(rng, "i8row" if kv == 8 else "f16", 1, sum(-(-n // page) for n in lengths) + 1, page, kv, d, rows, width, lengths)
    g = OnGpu(c)
    q = queries(rng, rows, kv * group, d)
    for bound in (longest, 3 * longest + 7, max(1, longest // 5)):
        check(g, q, d ** -0.5, max_length=bound)


@pytest.mark.parametrize("longest", [300, 2000, 9000, 50000])
def test_a_nan_in_one_part_reaches_its_heads_alone(longest):
    announce(f"attend NaN in a part, {longest} tokens")
    rng = rng_of(18, longest)
    c = Cache(rng, "f16", 1, -(-longest // 64) * 2, 64, 2, 64, 2, -(-longest // 64), [longest, longest - 5])
    at = c.table[0, (longest // 3) // 64]
    c.k[0, at, 1, (longest // 3) % 64, 5] = np.nan
    g = OnGpu(c)
    q = queries(rng, 2, 6, 64)
    y = attend(g, 0, q, 0.125)
    assert np.isnan(y[0, 3:]).all() and not np.isnan(y[0, :3]).any() and not np.isnan(y[1]).any()
    c.k[0, at, 1, (longest // 3) % 64, 5] = -np.inf   # scores of +inf or -inf by the sign of q
    g = OnGpu(c)
    y = attend(g, 0, q, 0.125)
    for h in range(3, 6):
        assert np.isnan(y[0, h]).all() if q[0, h, 5] < 0 else not np.isnan(y[0, h]).any()
