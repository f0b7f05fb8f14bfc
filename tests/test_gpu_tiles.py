"""Every kernel behind the 8-bit and expert products, in shapes that take it
(held against the library's rule by test_tile_choice.py): several tiles for a
workgroup, each way that an expert's rows can end, gathered and not, repeated
calls with the same bits."""
from __future__ import annotations

import pytest

import dequantize_mat_vec_amd as dmv
import tile_choice as choice
import tile_reference as ref
import tile_shapes as shapes
from gpu_util import announce, torch_dev

pytestmark = pytest.mark.gpu

GUARD, CANARY = 64, -12345.0
TOKENS = 61


def made(seed):
    torch, dev = torch_dev()
    gen = torch.Generator(device=dev).manual_seed(seed)

    def codes(*shape):
        return torch.randint(-128, 128, shape, generator=gen, device=dev, dtype=torch.int8)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev)

    def scales(size, *shape):
        return (torch.rand(shape, generator=gen, device=dev) + 0.5) * size

    def below(n, count):
        return torch.randint(0, max(n, 1), (count,), generator=gen, device=dev, dtype=torch.int32)
    return torch, dev, codes, normal, scales, below


class Experts:
    """Inputs of a call and its reference; rows of Y before the first and behind the last expert's."""

    def __init__(self, counts, n, k, form, gated, gather, seed, lead=1, behind=2):
        torch, dev, codes, normal, scales, below = made(seed)
        self.n, self.k, self.form, self.gated, self.e = n, k, form, gated, len(counts)
        self.starts = [lead]
        for c in counts:
            self.starts.append(self.starts[-1] + c)
        self.rows = self.starts[-1] + behind
        self.offsets = torch.tensor(self.starts, dtype=torch.int32, device=dev)
        tokens = TOKENS if gather else self.rows + 5
        self.at = None
        if gather:   # some indexes outside X
            self.at = below(tokens, self.rows)
            wild = torch.tensor([-1, tokens, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32, device=dev)
            self.at[::7] = wild[below(4, len(self.at[::7])).long()]
        mats = 2 if gated else 1
        if form == "f16":
            self.x, self.xs = normal(tokens, k).half(), None
            self.w, self.ws = [(normal(self.e, n, k) * 0.05).half() for _ in range(mats)], [None] * mats
        else:
            self.x, self.xs = codes(tokens, k), scales(0.02, tokens)
            self.w, self.ws = [codes(self.e, n, k) for _ in range(mats)], [scales(1e-4, self.e, n) for _ in range(mats)]
        self.bias = None if gated else normal(self.e, n)
        at = self.at if gather else torch.arange(self.rows, dtype=torch.int32, device=dev)
        scaled = form != "f16"
        parts = [ref.grouped(self.starts, w, self.x, at, self.bias, ws, self.xs) for w, ws in zip(self.w, self.ws)]
        tols = [ref.tolerance(y, size, k, scaled) for y, size in parts]
        self.want, self.tol = ref.joined(parts[0][0], parts[1][0], *tols) if gated else (parts[0][0], tols[0])
        self.own = torch.zeros(self.rows, dtype=torch.bool, device=dev)
        self.own[lead:self.starts[-1]] = True

    def call(self, y):
        form = "f16" if self.form == "f16" else "i8row"
        if self.gated:
            dmv.pesti_gemm_experts_swiglu(form, self.rows, self.e, self.n, self.k, self.offsets, *self.w, len(self.x), self.x, y,
                                          gate_scales=self.ws[0], up_scales=self.ws[1], x_scales=self.xs, x_rows=self.at)
        else:
            dmv.pesti_gemm_experts(form, self.rows, self.e, self.n, self.k, self.offsets, self.w[0], len(self.x), self.x, y,
                                   bias=self.bias, w_scales=self.ws[0], x_scales=self.xs, x_rows=self.at)


def run(call, rows, n, dtype, times=3):
    """Y of a call between guards; the calls after the first have its bits."""
    torch, dev = torch_dev()
    first = None
    for _ in range(times):
        buf = torch.full((2 * GUARD + rows * n,), CANARY, dtype=dtype, device=dev)
        y = buf[GUARD:GUARD + rows * n].view(rows, n)
        call(y)
        torch.cuda.synchronize()
        assert bool((buf[:GUARD] == buf[0]).all()) and bool((buf[GUARD + rows * n:] == buf[0]).all()), "wrote outside Y"
        assert first is None or torch.equal(first, y), "another call, other bits"
        first = y
    return first


def check(got, want, tol, what):
    bad = ~((got.double() - want).abs() <= tol)
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} outside, first at {bad.nonzero()[0].tolist()}"


def check_experts(c, what):
    torch, _ = torch_dev()
    for dtype in (torch.float32, torch.float16):
        announce(f"{what} {dtype}")
        y = run(c.call, c.rows, c.n, dtype)
        tol = ref.rounded(c.want, c.tol, dtype == torch.float16)
        check(y[c.own], c.want[c.own], tol[c.own], what)
        canary = torch.tensor(CANARY, dtype=dtype, device=y.device)
        assert bool((y[~c.own] == canary).all()), "a row outside every expert was written"


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("form", shapes.FORMS)
@pytest.mark.parametrize("case", range(len(shapes.TILES)))
def test_tiles_of_experts(case, form, gated):
    name, counts, n, k = shapes.TILES[case]
    n = n // 2 if gated else n
    gather = k != 160
    check_experts(Experts(counts, n, k, form, gated, gather, 100 + case), f"tiles {name} {form} gated {gated} n{n} k{k}")


@pytest.mark.parametrize("case", range(len(shapes.ROWS)))
def test_few_rows(case):
    name, counts, n, gated = shapes.ROWS[case]
    if counts is None:
        return check_dense(name, shapes.ROWS_DENSE_M[n], n, shapes.SHORT_K["i8"] + shapes.LONG_K["i8"], case)
    for form in shapes.FORMS:
        for k in shapes.SHORT_K[form] + shapes.LONG_K[form]:
            check_experts(Experts(counts, n, k, form, gated, k % 64 == 32, 200 + case), f"{name} {form} gated {gated} n{n} k{k}")


def check_dense(name, m, n, ks, seed):
    for k in ks:
        torch, dev, codes, normal, scales, _ = made(300 + seed)
        x, w, xs, ws, bias = codes(m, k), codes(n, k), scales(0.02, m), scales(1e-4, n), normal(n)
        want, size = ref.grouped([0, m], w[None], x, torch.arange(m, device=dev), bias[None], ws[None], xs)
        for dtype in (torch.float32, torch.float16):
            announce(f"dense {name} m{m} n{n} k{k} {dtype}")
            y = run(lambda y: dmv.pesti_gemm_i8row_i8token(m, n, k, w, ws, x, xs, y, bias), m, n, dtype)
            check(y, want, ref.rounded(want, ref.tolerance(want, size, k, True), dtype == torch.float16), f"dense {name}")


@pytest.mark.parametrize("case", range(len(shapes.DENSE)))
def test_tiles_of_the_dense_product(case):
    name, m, n = shapes.DENSE[case]
    check_dense(name, m, n, (96, 608), case)


@pytest.mark.parametrize("form,tokens", [("f16", 65535), ("i8", 131071)])
@pytest.mark.parametrize("counts,n", [([2, 0, 3], 40), ([300, 1, 99], 3000)])
def test_picked_rows_up_to_the_last_that_32_bits_address(counts, n, form, tokens):
    """X of just under 4 GiB, its last rows among those picked: the rows kernel and tiles."""
    torch, dev, codes, normal, scales, below = made(7)
    k, e, rows = 32768, len(counts), sum(counts)
    starts = [0]
    for c in counts:
        starts.append(starts[-1] + c)
    at = below(tokens, rows)
    at[::2] = tokens - 1 - at[::2] % 9
    announce(f"far rows of X {form} {counts}")
    if form == "f16":
        x, xs, ws = torch.empty(tokens, k, dtype=torch.float16, device=dev), None, None
        for part in x.split(8192):
            part.copy_(normal(*part.shape))
        w = (normal(e, n, k) * 0.05).half()
    else:
        x, xs, w, ws = codes(tokens, k), scales(0.02, tokens), codes(e, n, k), scales(1e-4, e, n)
    want, size = ref.grouped(starts, w, x, at, None, ws, xs)
    offsets = torch.tensor(starts, dtype=torch.int32, device=dev)
    y = run(lambda y: dmv.pesti_gemm_experts(form if form == "f16" else "i8row", rows, e, n, k, offsets, w, tokens, x, y, w_scales=ws,
                                             x_scales=xs, x_rows=at), rows, n, torch.float32)
    check(y, want, ref.tolerance(want, size, k, form != "f16"), "far rows of X")


def test_rows_of_x_past_4_gib_without_an_index():
    """X of more than 4 GiB, row r of it for row r of Y: the last rows."""
    torch, dev, codes, normal, scales, _ = made(8)
    m, n, k = 140001, 72, 32768
    x, w, xs, ws = codes(m, k), codes(n, k), scales(0.02, m), scales(1e-4, n)
    announce("X past 4 GiB")
    y = run(lambda y: dmv.pesti_gemm_i8row_i8token(m, n, k, w, ws, x, xs, y), m, n, torch.float32, times=1)
    for at in (slice(0, 300), slice(131072 - 150, 131072 + 150), slice(m - 300, m)):
        rows = torch.arange(m, device=dev)[at]
        want, size = ref.grouped([0, len(rows)], w[None], x, rows, None, ws[None], xs)
        check(y[at], want, ref.tolerance(want, size, k, True), "far rows of X")


def test_one_call_on_two_streams():
    """The largest tiles on two streams at once, each with its own Y: the bits of a call alone."""
    torch, dev = torch_dev()
    name, counts, n, k = shapes.TILES[1]
    c = Experts(counts, n, k, "f16", False, True, 11)
    assert choice.kernel(c.rows, n, k, "f16", c.e) == name
    alone = run(c.call, c.rows, n, torch.float32, times=1)
    streams = [torch.cuda.Stream() for _ in range(2)]
    ys = [torch.full_like(alone, CANARY) for _ in streams]
    torch.cuda.synchronize()
    announce("largest tiles on two streams")
    for _ in range(3):
        for y, s in zip(ys, streams):
            with torch.cuda.stream(s):
                c.call(y)
    torch.cuda.synchronize()
    for y in ys:
        assert torch.equal(y, alone)


def test_tiles_captured_and_replayed():
    """The largest tiles in a graph, replayed while the rows of the experts change, with eager calls between: every
    replay has the eager call's bits."""
    torch, dev = torch_dev()
    _, counts, n, k = shapes.TILES[1]
    c = Experts(counts, n // 2, k, "i8", True, False, 12)
    y = torch.full((c.rows, c.n), CANARY, dtype=torch.float16, device=dev)
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        c.call(y)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=stream):
            c.call(y)
    for r in range(4):
        announce(f"largest tiles graph replay {r}")
        counts = counts[r:] + counts[:r]
        c.offsets.copy_(torch.tensor([1] + [1 + sum(counts[:i + 1]) for i in range(len(counts))], dtype=torch.int32))
        y.fill_(CANARY)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        replayed = y.clone()
        y.fill_(CANARY)
        c.call(y)
        torch.cuda.synchronize()
        assert torch.equal(replayed, y), r
