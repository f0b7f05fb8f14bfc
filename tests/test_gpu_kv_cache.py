"""The paged key-value cache on the GPU against its plain form: rows written,
pages taken, shared, given back, copied and compacted, with lists that name a
sequence twice or none, pools that run out, and pages that are not there."""
from __future__ import annotations

import numpy as np
import pytest

import dequantize_mat_vec_amd as dmv
from gpu_util import announce, to_dev
from kv_reference import Cache

pytestmark = pytest.mark.gpu


class OnGpu:
    """A Cache's arrays on the GPU and the structs over them."""

    def __init__(self, c):
        import torch
        self.c = c
        self.arrays = {n: None if getattr(c, n) is None else to_dev(getattr(c, n)) for n in
                       ("k", "v", "k_scales", "v_scales", "table", "lengths", "refs")}
        a = self.arrays
        self.cache = dmv.kv_cache(c.fmt, c.layers, c.pages, c.page_size, c.kv_heads, c.head_dim, a["k"], a["v"], a["k_scales"],
                                  a["v_scales"])
        self.table = dmv.kv_table(a["table"], a["lengths"], a["refs"])
        self.status = torch.full((1,), 77, dtype=torch.int32, device="cuda")
        n = dmv.pesti_cache_workspace_bytes(self.cache, self.table)
        assert n > 0
        self.workspace = torch.full((n,), 0x5A, dtype=torch.uint8, device="cuda")

    def same(self, loose=()):
        import torch
        torch.cuda.synchronize()
        for n, t in self.arrays.items():
            want = getattr(self.c, n)
            if want is None or n in loose:
                continue
            got = t.cpu().numpy()
            assert np.array_equal(got.view(np.uint8), np.ascontiguousarray(want).view(np.uint8)), n


def ints(*v):
    return to_dev(np.array(v, np.int32))


def rng_of(*key):
    return np.random.default_rng([72, *key])


FORMS = [("f16", 1, 32, 8), ("f16", 3, 64, 16), ("i8row", 2, 96, 32), ("i8row", 5, 256, 8), ("f16", 2, 160, 64)]


@pytest.mark.parametrize("fmt,kv,d,page", FORMS + [("f16", 2, 128, 16), ("i8row", 2, 128, 16), ("i8row", 1, 32, 8), ("i8row", 2, 64, 16),
                                                   ("f16", 1, 192, 8), ("f16", 1, 224, 8), ("i8row", 1, 224, 8)])
@pytest.mark.parametrize("kind", [np.float32, np.float16])
def test_append(fmt, kv, d, page, kind):
    announce(f"append {fmt} {kv}x{d} page {page} {kind.__name__}")
    rng = rng_of(1, d, page)
    lengths = [0, 1, page, page + 1, 3 * page - 1, 7]
    g = OnGpu(Cache(rng, fmt, 2, 24, page, kv, d, 6, 5, lengths))
    seq = [1, 2, 2, 3, 3, 4, 5, 4]
    pos = [0, page - 1, 0, page, 0, 3 * page - 2, 6, 1]
    x = (rng.standard_normal((8, 2 * kv * d + 16)) * np.exp(rng.standard_normal((8, 1)) * 6)).astype(kind)
    x[0, :kv * d] = 0   # a row of zeros
    dev = to_dev(x)
    k, v = dev[:, :kv * d], dev[:, kv * d:2 * kv * d]   # parts of a wider projection
    dmv.pesti_cache_append(g.cache, g.table, 1, 8, k, v, seq_ids=ints(*seq), positions=ints(*pos))
    g.c.append(1, x[:, :kv * d].reshape(8, kv, d), x[:, kv * d:2 * kv * d].reshape(8, kv, d), seq, pos)
    g.same()


@pytest.mark.parametrize("fmt", ["f16", "i8row"])
def test_append_by_default_goes_to_the_last_token_of_sequence_r(fmt):
    announce(f"append last token {fmt}")
    rng = rng_of(2)
    g = OnGpu(Cache(rng, fmt, 1, 12, 8, 2, 64, 4, 4, [9, 0, 8, 25]))
    x = rng.standard_normal((2, 4, 2, 64)).astype(np.float32)
    dmv.pesti_cache_append(g.cache, g.table, 0, 4, to_dev(x[0]).view(4, 128), to_dev(x[1]).view(4, 128))
    g.c.append(0, x[0], x[1], range(4), [n - 1 for n in (9, 0, 8, 25)])
    g.same()


def test_append_passes_over_rows_that_have_no_place():
    announce("append without a place")
    rng = rng_of(3)
    c = Cache(rng, "f16", 1, 6, 8, 1, 32, 3, 3, [10, 5, 0])
    c.table[0, 1] = 6          # past the pool
    c.table[1, 0] = -5
    g = OnGpu(c)
    seq, pos = [0, 0, 0, 0, 1, 2, -1, 3, 1000000, 0], [0, 9, 10, -1, 2, 0, 0, 0, 0, 2147483647]
    x = rng.standard_normal((2, 10, 1, 32)).astype(np.float32)
    dmv.pesti_cache_append(g.cache, g.table, 0, 10, to_dev(x[0]).view(10, 32), to_dev(x[1]).view(10, 32), seq_ids=ints(*seq),
                           positions=ints(*pos))
    g.c.append(0, x[0], x[1], seq, pos)
    g.same()
    assert np.array_equal(c.k[0, c.table[0, 0], 0, 0], x[0, 0, 0].astype(np.float16))   # the one row that has a place


def test_append_values_at_the_formats_ends():
    announce("append extreme values")
    rng = rng_of(4)
    rows = np.zeros((10, 1, 32), np.float32)
    rows[0, 0, :3] = 65504, 65520, -1e30      # binary16's largest, past it
    rows[1, 0, :3] = 6e-8, 2.9e-8, -3e-8      # around its smallest
    rows[2, 0, 5] = np.inf
    rows[3, 0, 6] = np.nan
    rows[4, 0, :2] = 1e-44, -2e-45            # a scale that is zero or a subnormal
    rows[5, 0, :4] = 127, 0.5, 1.5, -2.5      # ties go away from zero
    rows[6, 0, :2] = 3e38, -1.2e36
    rows[7] = rng.standard_normal((1, 32)) * 1e-38
    rows[8, 0, :3] = 2e-43, 1e-43, -5e-44
    rows[9] = 1.0 + 2.0 ** -11 * np.arange(32) / 4
    for fmt in ("f16", "i8row"):
        g = OnGpu(Cache(rng, fmt, 1, 2, 16, 1, 32, 1, 1, [10]))
        dmv.pesti_cache_append(g.cache, g.table, 0, 10, to_dev(rows).view(10, 32), to_dev(rows[::-1].copy()).view(10, 32),
                               seq_ids=ints(*[0] * 10), positions=ints(*range(10)))
        g.c.append(0, rows, rows[::-1], [0] * 10, range(10))
        got = {n: g.arrays[n].cpu().numpy() for n in ("k", "v")}
        for n in ("k", "v"):
            assert np.array_equal(got[n], getattr(g.c, n), equal_nan=True), (fmt, n)
        if fmt == "i8row":
            for n in ("k_scales", "v_scales"):
                assert np.array_equal(g.arrays[n].cpu().numpy(), getattr(g.c, n), equal_nan=True), n


def test_extend_takes_the_lowest_free_pages_in_list_order():
    announce("extend")
    rng = rng_of(5)
    g = OnGpu(Cache(rng, "f16", 1, 100, 8, 1, 32, 7, 12, [0, 5, 8, 9, 30, 16, 0]))
    for seq, counts in (([4, 0, 2], [1, 17, 8]), ([3, 3, 1, 9, -2], [7, 50, 3, 4, 5]), ([6, 5, 4], [-4, 0, 40]), ([1, 0, 2, 3], None)):
        dmv.pesti_cache_extend(g.cache, g.table, len(seq), ints(*seq), None if counts is None else ints(*counts), g.status)
        assert g.c.extend(seq, [1] * len(seq) if counts is None else counts) == 0 == int(g.status[0])
        g.same()
    dmv.pesti_cache_extend(g.cache, g.table, 7, None, None, g.status)
    g.c.extend(range(7), [1] * 7)
    g.same()


def test_extend_changes_nothing_where_pages_or_places_run_out():
    announce("extend without room")
    rng = rng_of(6)
    g = OnGpu(Cache(rng, "f16", 1, 9, 8, 1, 32, 4, 6, [20, 8, 3, 0]))
    for seq, counts, want in (([0, 1, 3], [5, 30, 9], 3), ([1, 2], [1, 46], -1), ([3], [49], -1), ([3, 0], [2147483647, 1], -1)):
        dmv.pesti_cache_extend(g.cache, g.table, len(seq), ints(*seq), ints(*counts), g.status)
        assert g.c.extend(seq, counts) == want == int(g.status[0])
        g.same()
    dmv.pesti_cache_extend(g.cache, g.table, 2, ints(1, 3), ints(16, 16), g.status)   # exactly what is left
    assert g.c.extend([1, 3], [16, 16]) == 0 == int(g.status[0])
    g.same()


@pytest.mark.parametrize("pages", [31, 32, 33, 32768, 32769, 70001])
def test_free_pages_are_found_anywhere_in_the_pool(pages):
    announce(f"extend in a pool of {pages}")
    rng = rng_of(7, pages)
    c = Cache(rng, "f16", 1, pages, 8, 1, 32, 3, pages, [])
    free = np.unique(np.concatenate([rng.integers(0, pages, 20), [pages - 1, 0]]))
    c.refs[:] = rng.integers(1, 4, pages)
    c.refs[free] = 0
    g = OnGpu(c)
    dmv.pesti_cache_extend(g.cache, g.table, 2, ints(2, 0), ints(8 * (len(free) - 1), 5), g.status)
    assert c.extend([2, 0], [8 * (len(free) - 1), 5]) == 0 == int(g.status[0])
    g.same()
    assert c.table[0, 0] == pages - 1


def test_many_sequences():
    announce("extend, fork and free 4096 sequences")
    rng = rng_of(8)
    c = Cache(rng, "f16", 1, 10000, 8, 1, 32, 4096, 3, [], shuffle=False)
    g = OnGpu(c)
    order = rng.permutation(4096)[:2000]
    counts = rng.integers(0, 20, 2000)
    dmv.pesti_cache_extend(g.cache, g.table, 2000, to_dev(order.astype(np.int32)), to_dev(counts.astype(np.int32)), g.status)
    assert c.extend(order, counts) == 0 == int(g.status[0])
    g.same()
    rest = np.setdiff1d(np.arange(4096), order)
    children = np.concatenate([rest, rest])[:4000]
    parents = order[rng.integers(0, 2000, 4000)]
    dmv.pesti_cache_fork(g.cache, g.table, 4000, to_dev(parents.astype(np.int32)), to_dev(children.astype(np.int32)), g.status,
                         g.workspace)
    assert c.fork(parents, children) == 0 == int(g.status[0])
    g.same()
    dmv.pesti_cache_free(g.cache, g.table, 4096)
    c.free(range(4096))
    g.same()
    assert not c.refs.any() and not c.lengths.any()


@pytest.mark.parametrize("fmt,kv,d,page", FORMS)
def test_fork(fmt, kv, d, page):
    announce(f"fork {fmt} {kv}x{d} page {page}")
    rng = rng_of(9, d)
    g = OnGpu(Cache(rng, fmt, 3, 40, page, kv, d, 12, 6, [2 * page + 3, page, 1, 0, 5 * page + page // 2, 0, 0, 0, 0, 0, 0, 0]))
    # a full last page, a child of an empty parent, a child named twice, one that is not empty, names of none, a parent that is a child
    parents = [0, 0, 1, 4, 3, 2, 0, 4, -1, 2, 5, 12]
    children = [5, 6, 7, 8, 9, 5, 2, 4, 10, 99, 11, 10]
    dmv.pesti_cache_fork(g.cache, g.table, len(parents), ints(*parents), ints(*children), g.status, g.workspace)
    assert g.c.fork(parents, children) == 0 == int(g.status[0])
    g.same()
    assert list(g.c.lengths[5:12]) == [2 * page + 3, 2 * page + 3, page, 5 * page + page // 2, 0, 0, 0]
    # given back, some twice
    dmv.pesti_cache_free(g.cache, g.table, 7, ints(5, 0, 5, 8, -3, 12, 3))
    g.c.free([5, 0, 5, 8, -3, 12, 3])
    g.same()


def test_fork_changes_nothing_where_pages_run_out():
    announce("fork without room")
    rng = rng_of(10)
    g = OnGpu(Cache(rng, "f16", 2, 8, 8, 1, 64, 6, 4, [17, 9, 8]))
    dmv.pesti_cache_fork(g.cache, g.table, 3, ints(0, 1, 0), ints(3, 4, 5), g.status, g.workspace)
    assert g.c.fork([0, 1, 0], [3, 4, 5]) == 1 == int(g.status[0])
    g.same()
    dmv.pesti_cache_fork(g.cache, g.table, 3, ints(2, 1, 0), ints(3, 4, 5), g.status, g.workspace)
    assert g.c.fork([2, 1, 0], [3, 4, 5]) == 0 == int(g.status[0])
    g.same()


def test_upkeep_passes_over_pages_that_are_not_there():
    announce("bad pages in the table")
    rng = rng_of(11)
    c = Cache(rng, "i8row", 2, 20, 8, 2, 32, 6, 4, [30, 12, 20])
    c.table[0, 1], c.table[1, 1], c.table[2, 0], c.table[2, 2] = 20, -1, 2147483647, -2147483648
    g = OnGpu(c)
    dmv.pesti_cache_fork(g.cache, g.table, 3, ints(0, 1, 2), ints(3, 4, 5), g.status, g.workspace)
    assert c.fork([0, 1, 2], [3, 4, 5]) == 0 == int(g.status[0])
    g.same()
    dmv.pesti_cache_free(g.cache, g.table, 2, ints(0, 5))
    c.free([0, 5])
    g.same()
    dmv.pesti_cache_compact(g.cache, g.table, g.status, g.workspace)
    assert c.compact() == int(g.status[0])
    g.same()


@pytest.mark.parametrize("fmt,kv,d,page", FORMS)
@pytest.mark.parametrize("pages", [40, 1500])
def test_compact(fmt, kv, d, page, pages):
    announce(f"compact {fmt} {kv}x{d} page {page}, {pages} pages")
    rng = rng_of(12, d, pages)
    if pages > 40 and kv * d * page > 4096:
        kv, d = 1, 32
    c = Cache(rng, fmt, 2, pages, page, kv, d, 9, 6, [3 * page, 1, 0, 2 * page + 1, page, 6 * page - 1, page - 1, 0, 0])
    assert c.fork([0, 5], [7, 8]) == 0
    c.free([1, 3])
    g = OnGpu(c)
    dmv.pesti_cache_compact(g.cache, g.table, g.status, g.workspace)
    live = c.compact()
    assert live == int(g.status[0]) == (c.refs > 0).sum() and (c.refs[:live] > 0).all()
    g.same()
    dmv.pesti_cache_compact(g.cache, g.table, g.status, g.workspace)   # nothing is left to move
    assert c.compact() == live == int(g.status[0])
    g.same()


@pytest.mark.parametrize("held", [0, 1, 33000, 65000])
def test_compact_of_large_pools(held):
    """More pages than a round of the plan sees, all, none or half of them held."""
    announce(f"compact 65000 pages, {held} held")
    rng = rng_of(13, held)
    c = Cache(rng, "f16", 1, 65000, 8, 1, 32, 2, 65000, [8 * held, 0] if held else [])
    g = OnGpu(c)
    dmv.pesti_cache_compact(g.cache, g.table, g.status, g.workspace)
    assert c.compact() == held == int(g.status[0])
    g.same()


@pytest.mark.parametrize("fmt,kv,d,page", FORMS)
def test_copy_pages(fmt, kv, d, page):
    announce(f"copy pages {fmt} {kv}x{d} page {page}")
    rng = rng_of(14, d)
    g = OnGpu(Cache(rng, fmt, 3, 20, page, kv, d, 1, 1, []))
    src, dst = [3, 4, 3, 20, -1, 7, 6], [0, 1, 2, 5, 9, 20, 6]
    dmv.pesti_cache_copy_pages(g.cache, len(src), ints(*src), ints(*dst))
    for a, b in zip(src, dst):
        if 0 <= a < 20 and 0 <= b < 20:
            g.c.copy_page(a, b)
    g.same()


def test_nothing_to_do():
    announce("cache calls without work")
    rng = rng_of(15)
    g = OnGpu(Cache(rng, "f16", 1, 4, 8, 1, 32, 2, 2, [5, 0]))
    dmv.pesti_cache_extend(g.cache, g.table, 0, None, None, None)
    dmv.pesti_cache_append(g.cache, g.table, 0, 0, None, None, x_format="f16")
    dmv.pesti_cache_free(g.cache, g.table, 0)
    dmv.pesti_cache_fork(g.cache, g.table, 0, None, None, None, None)
    dmv.pesti_cache_copy_pages(g.cache, 0, None, None)
    assert int(g.status[0]) == 77
    g.same()


def test_a_captured_beam_step():
    """free, fork, extend and append captured once and replayed: every replay equals the plain form's step."""
    announce("captured beam step")
    import torch
    rng = rng_of(16)
    c = Cache(rng, "f16", 2, 64, 8, 2, 32, 6, 10, [13, 20])
    g = OnGpu(c)
    x = to_dev(rng.standard_normal((2, 6, 64)).astype(np.float16))
    children, parents, everyone = ints(2, 3, 4, 5), ints(0, 0, 1, 1), ints(0, 1, 2, 3, 4, 5)

    def step():
        dmv.pesti_cache_free(g.cache, g.table, 4, children)
        dmv.pesti_cache_fork(g.cache, g.table, 4, parents, children, g.status, g.workspace)
        dmv.pesti_cache_extend(g.cache, g.table, 6, everyone, None, g.status)
        for layer in range(2):
            dmv.pesti_cache_append(g.cache, g.table, layer, 6, x[0], x[1], seq_ids=everyone)

    def plain(xs):
        c.free([2, 3, 4, 5])
        assert c.fork([0, 0, 1, 1], [2, 3, 4, 5]) == 0 and c.extend(range(6), [1] * 6) == 0
        for layer in range(2):
            c.append(layer, xs[0].reshape(6, 2, 32), xs[1].reshape(6, 2, 32), range(6), c.lengths - 1)

    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    g.same()   # capture ran nothing
    for i in range(12):
        new = rng.standard_normal((2, 6, 64)).astype(np.float16)
        x.copy_(to_dev(new))
        graph.replay()
        plain(new)
        assert int(g.status[0]) == 0
        g.same()


@pytest.mark.parametrize("power", [0, -100, -127, -138, 90])
def test_ties_into_8_bits(power):
    """Halves of a scale that is a power of two: exactly between two codes, away from zero, also where the scale is a
    subnormal; a last row of values a rounding beside them."""
    announce(f"append ties, scale 2^{power}")
    rng = rng_of(31, power + 200)
    g = OnGpu(Cache(rng, "i8row", 1, 8, 16, 2, 64, 1, 4, (50,)))
    x = (rng.integers(-253, 254, (40, 2, 64)) / 2).astype(np.float64)
    x[..., 0] = 127
    x = np.ldexp(x, power).astype(np.float32)
    beside = np.nextafter(x, np.float32(0))
    beside[..., 0] = x[..., 0]
    for v in (x, beside):
        seq, pos = np.zeros(40, np.int32), np.arange(5, 45, dtype=np.int32)
        dmv.pesti_cache_append(g.cache, g.table, 0, 40, to_dev(v.reshape(40, -1)), to_dev(-v.reshape(40, -1)), seq_ids=to_dev(seq),
                               positions=to_dev(pos))
        g.c.append(0, v, -v, seq, pos)
        g.same()
