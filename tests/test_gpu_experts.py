"""The 8-bit linear layer and the expert-grouped products against the float64
oracle, through the C ABI."""
from __future__ import annotations

import numpy as np
import pytest

import oracle
import dequantize_mat_vec_amd as dmv
from gpu_util import announce, to_dev, torch_dev

pytestmark = pytest.mark.gpu

GUARD = 64
EPS32, EPS16 = 2.0 ** -24, 2.0 ** -11   # half a step of float32 and binary16, relative
CANARY = -12345.0


def guarded(rows, n, kind):
    """(buffer, [rows][n] view between guards), filled with a number no product gives."""
    torch, dev = torch_dev()
    buf = torch.full((2 * GUARD + rows * n,), CANARY, dtype=torch.float32 if kind == "f32" else torch.float16, device=dev)
    return buf, buf[GUARD:GUARD + rows * n]


def read(buf, view, rows, n):
    torch, _ = torch_dev()
    torch.cuda.synchronize()
    edge = torch.cat([buf[:GUARD], buf[GUARD + rows * n:]])
    assert bool((edge == edge[0]).all()), "kernel wrote outside Y"
    return view.cpu().numpy().astype(np.float64).reshape(rows, n)


def close(got, want, tol, what):
    """|got - want| <= tol; and where Y is binary16, infinity where the value rounds to it."""
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} outside, worst {np.nanmax(np.abs(got - want) / tol):.3g} of the bound"


def rounding(y, kind):
    """The last rounding to Y's type: half a step, or half the smallest subnormal of binary16."""
    return EPS16 * np.abs(y) + 2.0 ** -25 if kind == "f16" else 0.0 * y


def i8_tolerance(y, size, kind):
    """fma(float(acc) * xs, ws, bias): the sum's and the product's rounding on the product, the fma's on the
    result, two more for second-order terms; 2^-126 where factors are subnormal."""
    t = 3 * EPS32 * size + EPS32 * np.abs(y) + 2.0 ** -126
    return t + (1 + EPS16) * rounding(np.abs(y) + t, kind)


def f16_tolerance(y, size, k, kind):
    """Products of binary16 are exact in float32; k + 1 additions each round by at most a step (the matrix cores
    may cut instead of rounding to nearest)."""
    t = (k + 2) * 2 * EPS32 * size + 2.0 ** -126
    return t + (1 + EPS16) * rounding(np.abs(y) + t, kind)


def codes(rng, *shape):
    return rng.integers(-128, 128, size=shape).astype(np.int8)


def scales(rng, *shape):
    return (rng.random(shape) * 0.01 + 1e-4).astype(np.float32)


# --- quantizer ----------------------------------------------------------------
def run_quant(x, kind):
    torch, dev = torch_dev()
    m, k = x.shape
    buf = torch.full((m * k + 2 * GUARD,), 99, dtype=torch.int8, device=dev)
    s = torch.full((m + 2,), CANARY, dtype=torch.float32, device=dev)
    dmv.pesti_quant_i8token(kind, m, k, to_dev(x) if k else None, buf[GUARD:GUARD + m * k] if k else None, s[1:m + 1])
    torch.cuda.synchronize()
    assert bool((buf[:GUARD] == 99).all()) and bool((buf[GUARD + m * k:] == 99).all()), "codes outside"
    s = s.cpu().numpy()
    assert s[0] == CANARY and s[-1] == CANARY, "scales outside"
    return buf[GUARD:GUARD + m * k].cpu().numpy().reshape(m, k), s[1:-1]


@pytest.mark.parametrize("kind", ["f16", "f32"])
@pytest.mark.parametrize("m,k", [(1, 32), (1, 896), (3, 96), (5, 4864), (2, 8224), (2, 32768), (1023, 160),
                                 (1025, 896), (1026, 2080), (1027, 4096), (1030, 4128), (7, 0)])
def test_quant_equals_the_oracle(kind, m, k):
    """Codes and scales bit for bit."""
    announce(f"quant {kind} m{m} k{k}")
    rng = np.random.default_rng([1, m, k, kind == "f16"])
    x = rng.standard_normal((m, k)) * np.exp(rng.normal(0, 3, size=(m, 1)))
    with np.errstate(over="ignore"):
        x = x.astype(np.float16 if kind == "f16" else np.float32)
    if m > 2 and k:
        x[1] = 0
    q, s = run_quant(x, kind)
    q_ref, s_ref = oracle.quantize_i8token(x)   # binary16 rows can have overflowed to infinity
    assert np.array_equal(s, s_ref, equal_nan=True)
    assert np.array_equal(q, q_ref)


@pytest.mark.parametrize("kind", ["f16", "f32"])
def test_quant_ties_and_neighbours(kind):
    """Quotients on and next to every border: with the row's maximum 127 * 2^j the scale is exactly 2^j and
    (q + 1/2) 2^j a tie, which goes away from zero; its neighbours go to the nearer side."""
    t = np.float16 if kind == "f16" else np.float32
    rows = []
    for j in (-6, 0, 3):
        half = ((np.arange(-127, 127) + 0.5) * 2.0 ** j).astype(t)
        for v in (half, np.nextafter(half, t(np.inf)), np.nextafter(half, t(-np.inf))):
            rows.append(np.concatenate([[127 * 2.0 ** j], v, [0.0]]).astype(t))
    x = np.stack(rows)
    announce(f"quant ties {kind}")
    q, s = run_quant(x, kind)
    q_ref, s_ref = oracle.quantize_i8token(x)
    assert np.array_equal(s, s_ref) and np.array_equal(q, q_ref)
    assert q[0, 127] == -1 and q[0, 128] == 1   # -1/2 and 1/2


def test_quant_extreme_magnitudes():
    """Subnormal rows, rows whose scale rounds to zero or has few bits, the largest floats."""
    rng = np.random.default_rng(5)
    x = np.concatenate([rng.standard_normal((3, 64)).astype(np.float32) * np.float32(f)
                        for f in (1e-38, 1e-40, 3e-43, 1e-44, 1e-30, 1e-31, 1e37)])
    x = np.concatenate([x, np.full((1, 64), np.finfo(np.float32).max, np.float32),
                        (rng.integers(-300, 300, size=(4, 64)) * 2.0 ** -149).astype(np.float32)])
    announce("quant extremes")
    q, s = run_quant(x, "f32")
    q_ref, s_ref = oracle.quantize_i8token(x)
    assert np.array_equal(s, s_ref) and np.array_equal(q, q_ref)


@pytest.mark.parametrize("kind", ["f16", "f32"])
def test_quant_of_rows_that_are_not_finite(kind):
    x = np.ones((1024 + 4, 96), np.float16 if kind == "f16" else np.float32)
    x[0, 5], x[1, 95], x[2, 0], x[3, 7] = np.inf, -np.inf, np.nan, np.nan
    announce(f"quant non-finite {kind}")
    for rows in (x, x[:5]):
        q, s = run_quant(rows, kind)
        assert np.isnan(s[:4]).all() and not q[:4].any()
        assert (q[4:] == 127).all() and np.isfinite(s[4:]).all()


# --- dense product -------------------------------------------------------------
def run_i8(q, s, w, ws, bias, kind, stream=None):
    m, k = q.shape
    n = len(ws)
    buf, y = guarded(m, n, kind)
    dmv.pesti_gemm_i8row_i8token(m, n, k, to_dev(w) if k else None, to_dev(ws), to_dev(q) if k else None, to_dev(s), y,
                                 None if bias is None else to_dev(bias), stream=stream)
    return read(buf, y, m, n)


@pytest.mark.parametrize("kind", ["f32", "f16"])
@pytest.mark.parametrize("m", [1, 2, 15, 16, 17, 32, 33, 63, 64, 65, 100, 128, 129, 257, 300])
@pytest.mark.parametrize("n,k", [(1, 32), (7, 96), (16, 64), (130, 224), (896, 896), (259, 4864)])
def test_gemm_i8(m, n, k, kind):
    announce(f"gemm_i8 {kind} m{m} n{n} k{k}")
    rng = np.random.default_rng([2, m, n, k])
    q, w, s, ws = codes(rng, m, k), codes(rng, n, k), scales(rng, m), scales(rng, n)
    bias = rng.standard_normal(n).astype(np.float32) if m % 2 else None
    y, size = oracle.gemm_i8(q, s, w, ws, bias)
    close(run_i8(q, s, w, ws, bias, kind), y, i8_tolerance(y, size, kind), "gemm_i8")


@pytest.mark.parametrize("m,n,k", [(4096, 896, 896), (1000, 2304, 768), (513, 4864, 896), (3, 50257, 768), (70, 20000, 160),
                                   (2048, 64, 32768), (1, 64, 32768)])
def test_gemm_i8_larger(m, n, k):
    announce(f"gemm_i8 m{m} n{n} k{k}")
    rng = np.random.default_rng([3, m, n, k])
    q, w, s, ws = codes(rng, m, k), codes(rng, n, k), scales(rng, m), scales(rng, n)
    y, size = oracle.gemm_i8(q, s, w, ws)
    close(run_i8(q, s, w, ws, None, "f32"), y, i8_tolerance(y, size, "f32"), "gemm_i8")


@pytest.mark.parametrize("kind", ["f32", "f16"])
@pytest.mark.parametrize("m,n,k", [(8064, 4096, 32), (8065, 4096, 32), (8193, 4096, 32), (1984, 4096, 160),
                                   (1985, 4096, 160), (1921, 4096, 160), (4160, 896, 288), (4161, 896, 288),
                                   (4097, 896, 288), (544, 2304, 96), (545, 2304, 96)])
def test_gemm_i8_rows_end_at_half_a_tile(m, n, k, kind):
    """The last rows are half a tile, one more, or one alone, in tiles of 256, 128 (by 256 and by 128 columns) and
    64 rows; the rows behind Y stay as they were."""
    announce(f"gemm_i8 ends {kind} m{m} n{n} k{k}")
    rng = np.random.default_rng([21, m, n])
    q, w, s, ws = codes(rng, m, k), codes(rng, n, k), scales(rng, m), scales(rng, n)
    y, size = oracle.gemm_i8(q, s, w, ws)
    close(run_i8(q, s, w, ws, None, kind), y, i8_tolerance(y, size, kind), "gemm_i8")


@pytest.mark.parametrize("m", [1, 50, 700])
def test_linear_layer_captured_and_replayed(m):
    """Quantizer and product in a graph on new tokens each time: every replay has the eager calls' bits."""
    torch, dev = torch_dev()
    rng = np.random.default_rng([22, m])
    n, k = 200, 352
    w, ws, bias = to_dev(codes(rng, n, k)), to_dev(scales(rng, n)), to_dev(rng.standard_normal(n).astype(np.float32))
    x = torch.empty(m, k, device=dev)
    q, s = torch.empty(m, k, dtype=torch.int8, device=dev), torch.empty(m, device=dev)
    y = torch.empty(m, n, device=dev)

    def run():
        dmv.pesti_quant_i8token("f32", m, k, x, q, s)
        dmv.pesti_gemm_i8row_i8token(m, n, k, w, ws, q, s, y, bias)
    x.normal_()
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        run()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=stream):
            run()
    for r in range(4):
        announce(f"linear graph m{m} replay {r}")
        x.copy_(to_dev(rng.standard_normal((m, k)).astype(np.float32)))
        y.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        replayed = y.clone()
        run()
        torch.cuda.synchronize()
        assert torch.equal(replayed, y), r


@pytest.mark.parametrize("m", [1, 40, 200])
def test_gemm_i8_sums_are_exact_at_the_limits(m):
    """The largest sums there are (128^2 * 32768 = 2^29), and unit scales: every output an integer, exact
    in float32 where the sum is a multiple of 2^14."""
    k, n = 32768, 48
    q, w = np.full((m, k), -128, np.int8), np.full((n, k), -128, np.int8)
    w[1::2] = 127
    one = np.ones
    y = run_i8(q, one(m, np.float32), w, one(n, np.float32), None, "f32")
    assert (y[:, ::2] == 2.0 ** 29).all() and (y[:, 1::2] == -128.0 * 127 * 32768).all()


@pytest.mark.parametrize("m", [1, 20, 50, 200])
def test_gemm_i8_without_columns_and_nan_rows(m):
    """k = 0 gives the bias; a row whose scale is NaN gives NaN and leaves the others."""
    rng = np.random.default_rng([4, m])
    bias = rng.standard_normal(70).astype(np.float32)
    q, s = np.zeros((m, 0), np.int8), np.ones(m, np.float32)
    assert np.array_equal(run_i8(q, s, np.zeros((70, 0), np.int8), scales(rng, 70), bias, "f32"), np.tile(bias.astype(np.float64), (m, 1)))
    q, w, s, ws = codes(rng, m, 64), codes(rng, 70, 64), scales(rng, m), scales(rng, 70)
    s[m // 2] = np.nan
    y = run_i8(q, s, w, ws, bias, "f32")
    ref, size = oracle.gemm_i8(q, s, w, ws, bias)
    rest = np.arange(m) != m // 2
    assert np.isnan(y[m // 2]).all()
    close(y[rest], ref[rest], i8_tolerance(ref, size, "f32")[rest], "rows beside a NaN row")


def test_gemm_i8_binary16_overflow_is_infinite():
    q, w = np.full((1, 64), 127, np.int8), np.full((4, 64), 127, np.int8)
    y = run_i8(q, np.ones(1, np.float32), w, np.ones(4, np.float32), None, "f16")
    assert np.isposinf(y).all()


# --- experts ----------------------------------------------------------------------
def routed(rng, counts, tokens, lead=0, behind=0, wild=False):
    """offsets and x_rows of experts with these row counts, `lead` rows before the first and `behind` after the
    last that belong to nobody; some indexes outside X if wild."""
    offsets = (np.concatenate([[0], np.cumsum(counts)]) + lead).astype(np.int32)
    rows = int(offsets[-1]) + behind
    at = rng.integers(0, max(tokens, 1), size=rows).astype(np.int32)
    if wild and rows:
        at[rng.integers(0, rows, size=max(1, rows // 7))] = rng.choice([-1, tokens, 2 ** 31 - 1, -2 ** 31])
    return offsets, at, rows


def experts_inputs(rng, form, e, n, k, tokens, mats=1):
    if form == "f16":
        x = rng.standard_normal((tokens, k)).astype(np.float16)
        return x, None, [((rng.standard_normal((e, n, k)) * 0.05).astype(np.float16), None) for _ in range(mats)]
    return codes(rng, tokens, k), scales(rng, tokens), [(codes(rng, e, n, k), scales(rng, e, n)) for _ in range(mats)]


def dev_of(v):
    return None if v is None or v.size == 0 else to_dev(v)


def run_experts(form, offsets, rows, x, xs, w, ws, kind, x_rows=None, bias=None, stream=None):
    e, n, k = w.shape
    buf, y = guarded(rows, n, kind)
    dmv.pesti_gemm_experts(form if form == "f16" else "i8row", rows, e, n, k, to_dev(offsets), dev_of(w), len(x), dev_of(x), y,
                           bias=dev_of(bias), w_scales=dev_of(ws), x_scales=dev_of(xs), x_rows=dev_of(x_rows), stream=stream)
    return read(buf, y, rows, n)


def run_swiglu(form, offsets, rows, x, xs, gate, up, kind, x_rows=None):
    e, n, k = gate[0].shape
    buf, h = guarded(rows, n, kind)
    dmv.pesti_gemm_experts_swiglu(form if form == "f16" else "i8row", rows, e, n, k, to_dev(offsets), dev_of(gate[0]), dev_of(up[0]),
                                  len(x), dev_of(x), h, gate_scales=dev_of(gate[1]), up_scales=dev_of(up[1]), x_scales=dev_of(xs),
                                  x_rows=dev_of(x_rows))
    return read(buf, h, rows, n)


def check_experts(got, offsets, rows, form, x, xs, w, ws, kind, x_rows=None, bias=None):
    y, size = oracle.gemm_experts(offsets, w, x, rows, x_rows, bias, ws, xs)
    k = w.shape[2]
    own = ~np.isnan(y[:, 0])
    tol = f16_tolerance(y, size, k, kind) if form == "f16" else i8_tolerance(y, size, kind)
    if form != "f16":   # sum |x w| bounds |sum x w|, which the derivation takes; one |product| is enough
        p, _ = oracle.gemm_experts(offsets, w, x, rows, x_rows, None, ws, xs)
        b = np.abs(y - p)
        tol = i8_tolerance(y, np.abs(p) + b, kind)
    close(got[own], y[own], tol[own], f"experts {form}")
    canary = np.float16(CANARY) if kind == "f16" else np.float32(CANARY)
    assert (got[~own] == canary).all(), "a row outside every expert was written"


def check_swiglu(got, offsets, rows, form, x, xs, gate, up, kind, x_rows=None):
    k = gate[0].shape[2]
    g, sg = oracle.gemm_experts(offsets, gate[0], x, rows, x_rows, None, gate[1], xs)
    u, su = oracle.gemm_experts(offsets, up[0], x, rows, x_rows, None, up[1], xs)
    eg, eu = ((f16_tolerance(g, sg, k, "f32"), f16_tolerance(u, su, k, "f32")) if form == "f16" else
              (i8_tolerance(g, np.abs(g), "f32"), i8_tolerance(u, np.abs(u), "f32")))
    h = oracle.silu(g) * u
    # |silu'| <= 1.1; e^-g within 2 steps, the sum, the quotient and the product half a step each: 8 half steps.
    # e^-g overflows past g = -88, where |silu| < 1e-36.
    tol = 1.1 * eg * np.abs(u) + np.abs(oracle.silu(g)) * eu + 2 * eg * eu + 8 * EPS32 * np.abs(h) + 1e-35 * (1 + np.abs(u))
    tol = tol + (1 + EPS16) * rounding(np.abs(h) + tol, kind)
    own = ~np.isnan(h[:, 0])
    close(got[own], h[own], tol[own], f"swiglu {form}")
    canary = np.float16(CANARY) if kind == "f16" else np.float32(CANARY)
    assert (got[~own] == canary).all(), "a row outside every expert was written"


COUNTS = {
    "one row": [1],
    "empty experts": [0, 3, 0, 0, 1, 0],
    "ends inside tiles": [17, 15, 1, 33, 16, 2],
    "one expert has all": [0, 300, 0],
    "more experts than lanes": [i % 3 for i in range(130)],
    "mean over 32": [70, 1, 64, 40],
    "mean over 64": [129, 127, 0, 200, 5],
    "mean over 128, ragged": [400, 3, 257, 0, 128],
    "nobody has rows": [0, 0, 0],
}


@pytest.mark.parametrize("form", ["f16", "i8"])
@pytest.mark.parametrize("n,k", [(33, 96), (256, 160), (130, 1056)])
@pytest.mark.parametrize("which", list(COUNTS))
def test_experts(which, n, k, form):
    rng = np.random.default_rng([6, len(which), n, k])
    counts, tokens = COUNTS[which], 37
    kind = "f16" if (n + len(which)) % 2 else "f32"
    announce(f"experts {form} {kind} {which} n{n} k{k}")
    x, xs, ((w, ws),) = experts_inputs(rng, form, len(counts), n, k, tokens)
    offsets, at, rows = routed(rng, counts, tokens, lead=len(which) % 4, behind=5, wild=len(which) % 2 == 0)
    bias = rng.standard_normal((len(counts), n)).astype(np.float32) if k == 96 else None
    got = run_experts(form, offsets, rows, x, xs, w, ws, kind, at, bias)
    check_experts(got, offsets, rows, form, x, xs, w, ws, kind, at, bias)


@pytest.mark.parametrize("form", ["f16", "i8"])
@pytest.mark.parametrize("n,k", [(33, 96), (136, 1056)])
@pytest.mark.parametrize("which", list(COUNTS))
def test_swiglu(which, n, k, form):
    rng = np.random.default_rng([7, len(which), n, k])
    counts, tokens = COUNTS[which], 29
    kind = "f16" if (n + len(which)) % 2 else "f32"
    announce(f"swiglu {form} {kind} {which} n{n} k{k}")
    x, xs, (gate, up) = experts_inputs(rng, form, len(counts), n, k, tokens, mats=2)
    offsets, at, rows = routed(rng, counts, tokens, lead=len(which) % 3, behind=3, wild=len(which) % 2 == 1)
    got = run_swiglu(form, offsets, rows, x, xs, gate, up, kind, at)
    check_swiglu(got, offsets, rows, form, x, xs, gate, up, kind, at)


@pytest.mark.parametrize("mean", [1, 20, 40, 70, 150, 300])
@pytest.mark.parametrize("e", [64, 65, 700, 1024])
def test_experts_by_the_hundred(e, mean):
    """Many experts of every mean row count (each kernel's look-up of tiles), columns of several tiles; rows of
    X repeat.  Few columns of K: the oracle's work stays small."""
    rng = np.random.default_rng([16, e, mean])
    counts = rng.integers(0, 2 * mean + 1, size=e)
    counts[rng.integers(0, e, size=e // 5)] = 0
    n, k = 40, 32
    x, xs, ((w, ws),) = experts_inputs(rng, "i8", e, n, k, 50)
    offsets, at, rows = routed(rng, counts, 50, lead=1, behind=2)
    announce(f"experts by the hundred {e} {mean} rows {rows}")
    got = run_experts("i8", offsets, rows, x, xs, w, ws, "f32", at)
    check_experts(got, offsets, rows, "i8", x, xs, w, ws, "f32", at)


@pytest.mark.parametrize("form", ["f16", "i8"])
@pytest.mark.parametrize("gated", [False, True])
def test_several_tiles_for_a_workgroup(form, gated):
    """More tiles than workgroups run at a time, in the kernels of every tile size: each workgroup takes several,
    of different experts and widths, with K from one step to many."""
    for case, (counts, n, k) in enumerate([([700, 300, 1, 513, 400], 2600, 32), ([300, 140, 260, 3, 129], 3999, 288),
                                           ([90, 70, 65, 128, 0, 127], 9000, 96), ([40, 64, 33, 50], 20001, 64),
                                           ([600, 520, 770], 2800, 576)]):
        rng = np.random.default_rng([17, case])
        e = len(counts)
        if gated:
            n //= 2
        x, xs, mats = experts_inputs(rng, form, e, n, k, 61, mats=2 if gated else 1)
        offsets, at, rows = routed(rng, counts, 61, lead=case % 2, behind=1, wild=case % 2 == 0)
        announce(f"several tiles {form} {gated} {case}")
        if gated:
            got = run_swiglu(form, offsets, rows, x, xs, mats[0], mats[1], "f16", at)
            check_swiglu(got, offsets, rows, form, x, xs, mats[0], mats[1], "f16", at)
        else:
            bias = rng.standard_normal((e, n)).astype(np.float32)
            got = run_experts(form, offsets, rows, x, xs, mats[0][0], mats[0][1], "f32", at, bias)
            check_experts(got, offsets, rows, form, x, xs, mats[0][0], mats[0][1], "f32", at, bias)


@pytest.mark.parametrize("form", ["f16", "i8"])
def test_experts_without_gather_or_columns_or_tokens(form):
    """x_rows left out (row r of X is row r of Y); k = 0 and an empty X give the bias."""
    rng = np.random.default_rng([8, form == "f16"])
    for counts in ([3, 0, 9], [90, 70], [300, 20]):
        rows = sum(counts)
        offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        announce(f"experts {form} no gather {counts}")
        x, xs, ((w, ws),) = experts_inputs(rng, form, len(counts), 70, 224, rows)
        check_experts(run_experts(form, offsets, rows, x, xs, w, ws, "f32"), offsets, rows, form, x, xs, w, ws, "f32")
        bias = rng.standard_normal((len(counts), 70)).astype(np.float32)
        want = bias.astype(np.float64)[oracle.expert_of_rows(offsets, rows)]
        assert np.array_equal(run_experts(form, offsets, rows, x[:, :0], xs, w[:, :, :0], ws, "f32", None, bias), want)
        at = np.zeros(rows, np.int32)
        assert np.array_equal(run_experts(form, offsets, rows, x[:0], None if xs is None else xs[:0], w, ws, "f32", at, bias), want)


@pytest.mark.parametrize("form", ["f16", "i8"])
def test_experts_with_wild_offsets_stay_inside(form):
    """Offsets outside 0..rows are held to it, a range that ends before it starts is empty."""
    rng = np.random.default_rng([9, form == "f16"])
    x, xs, ((w, ws),) = experts_inputs(rng, form, 4, 40, 96, 20)
    offsets = np.array([-7, 6, 6, 2 ** 31 - 1, -2 ** 31], np.int32)   # 0..6, none, 6..20, none
    announce(f"experts {form} wild offsets")
    check_experts(run_experts(form, offsets, 20, x, xs, w, ws, "f32"), offsets, 20, form, x, xs, w, ws, "f32")


@pytest.mark.parametrize("form", ["f16", "i8"])
@pytest.mark.parametrize("rows", [5, 100, 300])
def test_rows_beside_values_that_are_not_finite(form, rows):
    """One row of X and one row of one expert's W hold infinities and NaN (8 bits: scales): the outputs that
    they reach are not finite, all others are as without them."""
    rng = np.random.default_rng([10, rows])
    x, xs, ((w, ws),) = experts_inputs(rng, form, 2, 70, 160, rows)
    offsets = np.array([0, rows // 2, rows], np.int32)
    announce(f"experts {form} non-finite {rows}")
    clean = run_experts(form, offsets, rows, x, xs, w, ws, "f32")
    if form == "f16":
        x[1, 3], w[1, 69, 159] = np.nan, np.inf
    else:
        xs[1], ws[1, 69] = np.nan, np.inf
    got = run_experts(form, offsets, rows, x, xs, w, ws, "f32")
    hit = np.zeros_like(clean, bool)
    hit[1] = True
    hit[rows // 2:, 69] = True
    assert not np.isfinite(got[hit & (clean != 0)]).any()
    assert np.array_equal(got[~hit], clean[~hit])


def test_one_expert_equals_the_dense_product():
    """All rows in one expert: bit for bit the dense call's Y (integer sums, the same rounding)."""
    rng = np.random.default_rng(11)
    for m in (1, 17, 33, 64, 150):
        q, w, s, ws = codes(rng, m, 224), codes(rng, 100, 224), scales(rng, m), scales(rng, 100)
        a = run_i8(q, s, w, ws, None, "f32")
        b = run_experts("i8", np.array([0, m], np.int32), m, q, s, w[None], ws[None], "f32")
        assert np.array_equal(a, b), m


# --- used together ------------------------------------------------------------------
def moe(x, top, gate, up, down, form):
    """One expert feed-forward block: tokens sorted by expert, quantized once, gate and up joined, the result
    quantized, the down projection.  Every stage's buffers, on the device."""
    torch, dev = torch_dev()
    tokens, k = x.shape
    e, f, _ = gate[0].shape
    ids = torch.from_numpy(top.reshape(-1)).to(dev)
    order = torch.argsort(ids, stable=True)
    offsets = torch.cat([ids.new_zeros(1), torch.bincount(ids, minlength=e).cumsum(0)]).to(torch.int32)
    at = (order // top.shape[1]).to(torch.int32)
    rows = len(ids)
    xd = to_dev(x)
    h = torch.empty(rows, f, dtype=torch.float16, device=dev)
    y = torch.empty(rows, k, dtype=torch.float32, device=dev)
    q = torch.empty(tokens, k, dtype=torch.int8, device=dev)
    s = torch.empty(tokens, dtype=torch.float32, device=dev)
    hq = torch.empty(rows, f, dtype=torch.int8, device=dev)
    hs = torch.empty(rows, dtype=torch.float32, device=dev)
    dv = [(to_dev(a), dev_of(b)) for a, b in (gate, up, down)]

    def run():
        if form == "i8":
            dmv.pesti_quant_i8token("f16", tokens, k, xd, q, s)
            dmv.pesti_gemm_experts_swiglu("i8row", rows, e, f, k, offsets, dv[0][0], dv[1][0], tokens, q, h, dv[0][1], dv[1][1], s, at)
            dmv.pesti_quant_i8token("f16", rows, f, h, hq, hs)
            dmv.pesti_gemm_experts("i8row", rows, e, k, f, offsets, dv[2][0], rows, hq, y, w_scales=dv[2][1], x_scales=hs)
        else:
            dmv.pesti_gemm_experts_swiglu("f16", rows, e, f, k, offsets, dv[0][0], dv[1][0], tokens, xd, h, x_rows=at)
            dmv.pesti_gemm_experts("f16", rows, e, k, f, offsets, dv[2][0], rows, h, y)

    return run, dict(x=xd, offsets=offsets, at=at, h=h, y=y, q=q, s=s, hq=hq, hs=hs)


@pytest.mark.parametrize("form", ["f16", "i8"])
@pytest.mark.parametrize("tokens", [1, 40, 300])
def test_feed_forward_block_of_experts(tokens, form):
    """The calls in a row as a model makes them, each stage against the oracle on what the stage before it left."""
    torch, _ = torch_dev()
    rng = np.random.default_rng([12, tokens])
    e, f, k = 6, 160, 96
    top = np.stack([rng.permutation(e)[:2] for _ in range(tokens)])
    x = rng.standard_normal((tokens, k)).astype(np.float16)
    _, _, (gate, up) = experts_inputs(rng, form, e, f, k, 1, mats=2)
    _, _, (down,) = experts_inputs(rng, form, e, k, f, 1)
    announce(f"block {form} {tokens}")
    run, b = moe(x, top, gate, up, down, form)
    run()
    torch.cuda.synchronize()
    n = {name: t.cpu().numpy() for name, t in b.items()}
    rows = len(n["at"])
    if form == "i8":
        q, s = oracle.quantize_i8token(x)
        assert np.array_equal(n["q"], q) and np.array_equal(n["s"], s)
        check_swiglu(n["h"].astype(np.float64), n["offsets"], rows, form, q, s, gate, up, "f16", n["at"])
        q, s = oracle.quantize_i8token(n["h"])
        assert np.array_equal(n["hq"], q) and np.array_equal(n["hs"], s)
        check_experts(n["y"].astype(np.float64), n["offsets"], rows, form, q, s, *down, "f32")
    else:
        check_swiglu(n["h"].astype(np.float64), n["offsets"], rows, form, x, None, gate, up, "f16", n["at"])
        check_experts(n["y"].astype(np.float64), n["offsets"], rows, form, n["h"], None, *down, "f32")


@pytest.mark.parametrize("form", ["f16", "i8"])
def test_block_captured_and_replayed(form):
    """The block in a graph, replayed while the tokens, the routing and its row counts change: every replay has
    the eager calls' bits."""
    torch, dev = torch_dev()
    rng = np.random.default_rng(13)
    tokens, e, f, k = 48, 5, 96, 64
    x = rng.standard_normal((tokens, k)).astype(np.float16)
    _, _, (gate, up) = experts_inputs(rng, form, e, f, k, 1, mats=2)
    _, _, (down,) = experts_inputs(rng, form, e, k, f, 1)
    top = np.stack([rng.permutation(e)[:2] for _ in range(tokens)])
    run, b = moe(x, top, gate, up, down, form)
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        run()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=stream):
            run()
    for r in range(4):
        announce(f"block graph {form} replay {r}")
        top = np.stack([rng.permutation(e if r % 2 else 2)[:2] for _ in range(tokens)])   # other experts stay empty
        ids = torch.from_numpy(top.reshape(-1)).to(dev)
        b["at"].copy_((torch.argsort(ids, stable=True) // 2).to(torch.int32))
        b["offsets"].copy_(torch.cat([ids.new_zeros(1), torch.bincount(ids, minlength=e).cumsum(0)]).to(torch.int32))
        b["x"].copy_(to_dev(rng.standard_normal((tokens, k)).astype(np.float16)))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        replayed = {name: b[name].clone() for name in ("h", "y")}
        run()
        torch.cuda.synchronize()
        for name, t in replayed.items():
            assert torch.equal(t, b[name]), (r, name)


def test_calls_on_two_streams():
    """The same calls on two streams at once, each with its own buffers, have the bits of calls made one by one."""
    torch, _ = torch_dev()
    rng = np.random.default_rng(14)
    made = []
    for form, tokens in (("i8", 200), ("f16", 170)):
        e, f, k = 4, 224, 160
        top = np.stack([rng.permutation(e)[:2] for _ in range(tokens)])
        _, _, (gate, up) = experts_inputs(rng, form, e, f, k, 1, mats=2)
        _, _, (down,) = experts_inputs(rng, form, e, k, f, 1)
        made.append(moe(rng.standard_normal((tokens, k)).astype(np.float16), top, gate, up, down, form))
    for run, _ in made:
        run()
    torch.cuda.synchronize()
    want = [b["y"].clone() for _, b in made]
    for _, b in made:
        b["y"].zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in made]
    announce("two streams")
    for _ in range(5):
        for (run, _), st in zip(made, streams):
            with torch.cuda.stream(st):
                run()
    torch.cuda.synchronize()
    for (_, b), w in zip(made, want):
        assert torch.equal(b["y"], w)


def test_matrices_and_outputs_past_32_bit_offsets():
    """Experts whose matrices start past 4 GB, and Y past 4 GB: the last expert's and the last rows."""
    torch, dev = torch_dev()
    rng = np.random.default_rng(15)
    e, n, k, rows = 10, 16384, 32768, 20
    gen = torch.Generator(device="cuda").manual_seed(1)
    w = torch.randint(-128, 128, (e, n, k), generator=gen, device=dev, dtype=torch.int8)
    ws, x, xs = scales(rng, e, n), codes(rng, rows, k), scales(rng, rows)
    offsets = np.array([0] * 9 + [7, rows], np.int32)   # experts 8 and 9
    y = torch.zeros(rows, n, device=dev)
    announce("W past 4 GB")
    dmv.pesti_gemm_experts("i8row", rows, e, n, k, to_dev(offsets), w, rows, to_dev(x), y, w_scales=to_dev(ws), x_scales=to_dev(xs))
    torch.cuda.synchronize()
    for ex, a, b in ((8, 0, 7), (9, 7, rows)):
        for c0 in (0, n - 256):
            ref, size = oracle.gemm_i8(x[a:b], xs[a:b], w[ex, c0:c0 + 256].cpu().numpy(), ws[ex, c0:c0 + 256])
            close(y[a:b, c0:c0 + 256].cpu().numpy().astype(np.float64), ref, i8_tolerance(ref, size, "f32"), "far W")
    del w
    m, n, k = 70001, 32768, 32
    q, s, wc, ws = codes(rng, m, k), scales(rng, m), codes(rng, n, k), scales(rng, n)
    y = torch.zeros(m, n, dtype=torch.float16, device=dev)
    announce("Y past 4 GB")
    dmv.pesti_gemm_i8row_i8token(m, n, k, to_dev(wc), to_dev(ws), to_dev(q), to_dev(s), y)
    torch.cuda.synchronize()
    for at in (slice(0, 40), slice(m - 40, m)):
        ref, size = oracle.gemm_i8(q[at], s[at], wc, ws)
        close(y[at].cpu().numpy().astype(np.float64), ref, i8_tolerance(ref, size, "f16"), "far Y")


def test_binding_checks_sizes_and_types():
    torch, dev = torch_dev()
    t = lambda dtype, n: torch.zeros(n, dtype=dtype, device=dev)  # noqa: E731
    i8, f32, i32, i64 = torch.int8, torch.float32, torch.int32, torch.int64
    with pytest.raises(ValueError, match="offsets"):
        dmv.pesti_gemm_experts("i8row", 4, 2, 32, 32, t(i64, 3), t(i8, 2048), 4, t(i8, 128), t(f32, 128), w_scales=t(f32, 64),
                               x_scales=t(f32, 4))
    with pytest.raises(ValueError, match="x_rows"):
        dmv.pesti_gemm_experts("i8row", 4, 2, 32, 32, t(i32, 3), t(i8, 2048), 4, t(i8, 128), t(f32, 128), w_scales=t(f32, 64),
                               x_scales=t(f32, 4), x_rows=t(i32, 3))
    with pytest.raises(ValueError, match="w holds"):
        dmv.pesti_gemm_experts("f16", 4, 2, 32, 32, t(i32, 3), t(i8, 2048), 4, t(torch.float16, 128), t(f32, 128))
    with pytest.raises(ValueError, match="y holds"):
        dmv.pesti_gemm_i8row_i8token(4, 32, 32, t(i8, 1024), t(f32, 32), t(i8, 128), t(f32, 4), t(f32, 127))
    with pytest.raises(ValueError, match="contiguous"):
        dmv.pesti_quant_i8token("f32", 4, 32, t(f32, 256).view(4, 64)[:, :32], t(i8, 128), t(f32, 4))
