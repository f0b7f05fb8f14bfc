"""4-bit mat-vecs with group scales on the GPU against the 64-bit form: group
sizes, row lengths and counts that end anywhere in a tile, zero points, batches,
grouped and paired launches, magnitudes and non-finite values of x."""
from __future__ import annotations

import numpy as np
import pytest

import dequantize_mat_vec_amd as dmv
from gpu_util import announce, guarded_y, guards_intact, to_dev
from kv_reference import i4_matrix, i4_tolerance, i4_weights, silu

pytestmark = pytest.mark.gpu


def case_rng(*key):
    return np.random.default_rng([71, *key])


def put(m):
    packed, scales, zeros = m
    return to_dev(packed), to_dev(scales), None if zeros is None else to_dev(zeros)


def run(m, out, inf, group, x, bias=None, stream=None):
    import torch
    batch = x.shape[0]
    buf, y = guarded_y(batch * out)
    p, s, z = put(m)
    dmv.pesti_gemv_i4group(out, inf, group, p, s, z, to_dev(x), y, None if bias is None else to_dev(bias), batch, stream)
    torch.cuda.synchronize()
    assert guards_intact(buf, batch * out)
    return y.cpu().numpy().reshape(batch, out).astype(np.float64)


def check(m, out, inf, group, x, bias=None):
    w = i4_weights(*m, inf, group)
    exact = x.astype(np.float64) @ w.T
    tol = i4_tolerance(w, x.astype(np.float64))
    if bias is not None:
        exact = exact + bias.astype(np.float64)
        tol = tol + 2.0 ** -23 * np.abs(bias)
    y = run(m, out, inf, group, x, bias)
    err = np.abs(y - exact)
    assert np.all(err <= tol + 2.0 ** -24 * np.abs(exact)), (float((err / tol).max()), int(np.argmax(err / tol)))


# rows ends: within a 16-row tile, at it, behind it; lengths: one 32-weight step, short last chunks, several phases
SHAPES = [(1, 32, 32), (15, 64, 32), (16, 96, 64), (17, 128, 128), (33, 160, 32), (40, 896, 128), (97, 896, 32), (64, 928, 64),
          (31, 1056, 256), (48, 4864, 128), (20, 4096, 64), (7, 5024, 512), (5, 8192, 32), (3, 14336, 128), (4, 16416, 32768),
          (2, 32768, 64), (300, 224, 32), (1200, 288, 64), (4099, 256, 128)]


@pytest.mark.parametrize("out,inf,group", SHAPES)
@pytest.mark.parametrize("batch", [1, 3, 8])
def test_shapes(out, inf, group, batch):
    announce(f"i4group {batch}x{out}x{inf} group {group}")
    rng = case_rng(out, inf, group, batch)
    x = rng.standard_normal((batch, inf)).astype(np.float32)
    bias = rng.standard_normal(out).astype(np.float32) if batch != 3 else None
    check(i4_matrix(rng, out, inf, group, zeros=batch != 1), out, inf, group, x, bias)


@pytest.mark.parametrize("batch", range(1, 9))
def test_every_batch(batch):
    announce(f"i4group batch {batch}")
    rng = case_rng(1, batch)
    check(i4_matrix(rng, 83, 640, 64), 83, 640, 64, rng.standard_normal((batch, 640)).astype(np.float32))


# tall matrices, where workgroups take several tiles in turn
@pytest.mark.parametrize("batch,out,inf,group", [(1, 40001, 256, 128), (8, 20011, 896, 64), (2, 70003, 96, 32), (5, 33000, 1184, 32),
                                                 (8, 17000, 2080, 128)])
def test_tall(batch, out, inf, group):
    announce(f"i4group tall {batch}x{out}x{inf} group {group}")
    rng = case_rng(2, out)
    check(i4_matrix(rng, out, inf, group), out, inf, group, rng.standard_normal((batch, inf)).astype(np.float32),
          rng.standard_normal(out).astype(np.float32))


def test_zero_points_of_any_value():
    announce("i4group zero points")
    rng = case_rng(3)
    packed, scales, _ = i4_matrix(rng, 50, 512, 32)
    zeros = rng.integers(0, 256, scales.shape, dtype=np.uint8)
    zeros[:8] = np.array([0, 15, 16, 127, 128, 200, 254, 255], np.uint8)[:, None]
    check((packed, scales, zeros), 50, 512, 32, rng.standard_normal((4, 512)).astype(np.float32))


def test_rows_of_zero_weights_give_the_bias():
    announce("i4group zero weights")
    rng = case_rng(4)
    packed, scales, zeros = i4_matrix(rng, 40, 896, 128)
    packed[5:20] = 0x99   # every code 9
    zeros[5:20] = 9
    x, bias = rng.standard_normal((2, 896)).astype(np.float32), rng.standard_normal(40).astype(np.float32)
    y = run((packed, scales, zeros), 40, 896, 128, x, bias)
    assert np.array_equal(y[:, 5:20].astype(np.float32), np.broadcast_to(bias[5:20], (2, 15)))


@pytest.mark.parametrize("size", [1e-38, 1e-20, 1e-5, 1.0, 3e4, 1e10, 1e30])
def test_magnitudes_of_x(size):
    announce(f"i4group x of {size}")
    rng = case_rng(5)
    x = (rng.standard_normal((2, 384)) * size).astype(np.float32)
    check(i4_matrix(rng, 37, 384, 64), 37, 384, 64, x)


def test_wide_range_within_a_row():
    """One element 2^27 times the others, on a zero weight: the others keep their bits."""
    announce("i4group wide range")
    rng = case_rng(6)
    packed, scales, zeros = i4_matrix(rng, 32, 256, 32)
    packed[:, 8] = (packed[:, 8] & 0xF0) | 7   # weight 16
    zeros[:, 0] = 7
    x = rng.standard_normal((1, 256)).astype(np.float32)
    x[0, 16] = 2.0 ** 27
    check((packed, scales, zeros), 32, 256, 32, x)


def test_not_finite():
    """An infinity or NaN in one column reaches that column alone, as the sum of its products."""
    announce("i4group infinities and NaN")
    rng = case_rng(7)
    m = i4_matrix(rng, 35, 320, 32)
    packed, scales, zeros = m
    zeros[:] = 20   # no weight is zero, all of one sign
    x = rng.standard_normal((4, 320)).astype(np.float32)
    x[1, 77], x[2, 5], x[2, 6] = np.inf, np.inf, -np.inf
    x[3, 300] = np.nan
    y = run(m, 35, 320, 32, x)
    w = i4_weights(*m, 320, 32)
    exact = x[0].astype(np.float64) @ w.T
    assert np.all(np.abs(y[0] - exact) <= i4_tolerance(w, x[:1].astype(np.float64))[0] + 2.0 ** -24 * np.abs(exact))
    assert np.all(y[1] == -np.inf) and np.isnan(y[2]).all() and np.isnan(y[3]).all()


def test_scales_of_every_kind():
    announce("i4group scales")
    rng = case_rng(8)
    packed, scales, zeros = i4_matrix(rng, 32, 512, 64)
    scales[0], scales[1], scales[2], scales[3] = 0, -0.5, 6e-8, 65504
    x = rng.standard_normal((3, 512)).astype(np.float32)
    check((packed, scales, zeros), 32, 512, 64, x)


def test_padding_bytes_are_not_read_into_the_result():
    """A matrix at the end of its memory, rows and groups that do not fill a tile: what lies around does not matter."""
    announce("i4group surroundings")
    import torch
    rng = case_rng(9)
    out, inf, group = 21, 352, 64
    m = i4_matrix(rng, out, inf, group)
    x = rng.standard_normal((2, inf)).astype(np.float32)
    ys = []
    for fill in (0, 255):
        dev = []
        for a in m:
            a = np.ascontiguousarray(a)
            whole = torch.full((a.nbytes + 512,), fill, dtype=torch.uint8, device="cuda")
            whole[256:256 + a.nbytes] = torch.from_numpy(a.reshape(-1).view(np.uint8)).cuda()
            dev.append(whole[256:256 + a.nbytes])
        y = torch.empty(2, out, device="cuda")
        dmv.pesti_gemv_i4group(out, inf, group, dev[0], dev[1].view(torch.float16), dev[2], to_dev(x), y, None, 2)
        ys.append(y.cpu())
    assert torch.equal(*ys)
    w = i4_weights(*m, inf, group)
    assert np.all(np.abs(ys[0].numpy() - x.astype(np.float64) @ w.T) <= 2 * i4_tolerance(w, x.astype(np.float64)))


@pytest.mark.parametrize("group", [32, 64, 128, 1024])
@pytest.mark.parametrize("batch", [1, 5])
def test_grouped_launch_has_the_bits_of_single_calls(group, batch):
    announce(f"i4group grouped launch, groups of {group}, batch {batch}")
    import torch
    rng = case_rng(10, group)
    ops, singles, shapes = [], [], [(896, 896), (128, 896), (130, 416), (1, 32), (40, 0), (0, 64), (5000, 96), (33, 4864)]
    keep = []
    for i, (out, inf) in enumerate(shapes):
        p, s, z = put(i4_matrix(rng, out, inf, group, zeros=i % 2 == 0))
        x = to_dev(rng.standard_normal((batch, inf)).astype(np.float32))
        b = to_dev(rng.standard_normal(out).astype(np.float32)) if i % 3 else None
        y, y1 = (torch.full((batch, out), 7.0, device="cuda") for _ in range(2))
        ops.append((out, inf, p, s, z, x, y, b))
        dmv.pesti_gemv_i4group(out, inf, group, p, s, z, x, y1, b, batch)
        singles.append(y1)
        keep.append((p, s, z, x, b))
    dmv.pesti_gemv_group_i4group(ops, group, batch)
    torch.cuda.synchronize()
    for op, y1 in zip(ops, singles):
        assert torch.equal(op[6], y1), op[:2]


def test_empty_rows_and_no_columns():
    announce("i4group empty")
    import torch
    y = torch.full((2, 5), 7.0, device="cuda")
    b = torch.arange(5.0, device="cuda")
    dmv.pesti_gemv_i4group(5, 0, 32, None, None, None, None, y, b, 2)
    assert torch.equal(y, b.expand(2, 5))
    dmv.pesti_gemv_i4group(5, 0, 32, None, None, None, None, y, None, 2)
    assert torch.equal(y, torch.zeros(2, 5, device="cuda"))
    y.fill_(7.0)
    dmv.pesti_gemv_i4group_swiglu(5, 0, 32, None, None, None, None, None, None, None, y, 2)
    assert torch.equal(y, torch.zeros(2, 5, device="cuda"))
    y.fill_(7.0)
    dmv.pesti_gemv_i4group(0, 64, 32, None, None, None, None, None, None, 2)
    dmv.pesti_gemv_i4group(5, 64, 32, None, None, None, None, None, None, 0)
    assert torch.equal(y, torch.full((2, 5), 7.0, device="cuda"))


@pytest.mark.parametrize("batch,out,inf,group", [(1, 4864, 896, 128), (1, 33, 96, 32), (2, 17, 4128, 64), (8, 200, 5120, 32),
                                                 (5, 3001, 1024, 64), (3, 20000, 512, 256), (4, 6, 16384, 128)])
@pytest.mark.parametrize("zeros", [True, False])
def test_swiglu(batch, out, inf, group, zeros):
    announce(f"i4group swiglu {batch}x{out}x{inf} group {group} zeros {zeros}")
    import torch
    rng = case_rng(11, out)
    gate, up = (i4_matrix(rng, out, inf, group, zeros) for _ in range(2))
    x = rng.standard_normal((batch, inf)).astype(np.float32)
    buf, h = guarded_y(batch * out)
    dmv.pesti_gemv_i4group_swiglu(out, inf, group, *put(gate), *put(up), to_dev(x), h, batch)
    torch.cuda.synchronize()
    assert guards_intact(buf, batch * out)
    wg, wu, x = i4_weights(*gate, inf, group), i4_weights(*up, inf, group), x.astype(np.float64)
    g, u, eg, eu = x @ wg.T, x @ wu.T, i4_tolerance(wg, x), i4_tolerance(wu, x)
    # silu's slope is at most 1.1; the exponential, quotient and product add a few roundings of the result
    tol = 1.1 * eg * (np.abs(u) + eu) + np.abs(silu(g)) * eu + 2.0 ** -20 * np.abs(silu(g) * u) + 1e-30
    err = np.abs(h.cpu().numpy().reshape(batch, out) - silu(g) * u)
    assert np.all(err <= tol), float((err / tol).max())


@pytest.mark.parametrize("rows,inf,group", [(1, 32, 32), (37, 896, 128), (5, 160, 64), (300, 4864, 32), (3, 96, 32768)])
@pytest.mark.parametrize("zeros", [True, False])
def test_dequant_is_exact(rows, inf, group, zeros):
    announce(f"i4group dequant {rows}x{inf} group {group} zeros {zeros}")
    import torch
    rng = case_rng(12, rows)
    m = i4_matrix(rng, rows, inf, group, zeros)
    if zeros:
        m = (m[0], m[1], rng.integers(0, 256, m[1].shape, dtype=np.uint8))
    buf, w = guarded_y(rows * inf)
    dmv.pesti_dequant_i4group(rows, inf, group, *put(m), w)
    torch.cuda.synchronize()
    assert guards_intact(buf, rows * inf)
    assert np.array_equal(w.cpu().numpy().reshape(rows, inf).astype(np.float64), i4_weights(*m, inf, group))


def test_other_stream_and_captured_graph():
    announce("i4group stream and graph")
    import torch
    rng = case_rng(13)
    out, inf, group, batch = 500, 896, 64, 4
    p, s, z = put(i4_matrix(rng, out, inf, group))
    xs = [to_dev(rng.standard_normal((batch, inf)).astype(np.float32)) for _ in range(4)]
    eager = []
    for x in xs:
        y = torch.empty(batch, out, device="cuda")
        dmv.pesti_gemv_i4group(out, inf, group, p, s, z, x, y, None, batch)
        eager.append(y)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    y = torch.empty(batch, out, device="cuda")
    x = xs[0].clone()
    torch.cuda.synchronize()
    dmv.pesti_gemv_i4group(out, inf, group, p, s, z, x, y, None, batch, stream=side)
    side.synchronize()
    assert torch.equal(y, eager[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dmv.pesti_gemv_i4group(out, inf, group, p, s, z, x, y, None, batch)
    for i in (1, 2, 3, 0):
        x.copy_(xs[i])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, eager[i])


# how the work is dealt out by size: x whole in LDS with one or two buffers of sums, in phases with one to eight tiles
# of a workgroup (the last with fewer, and more workgroups than compute units), few rows by single wavefronts
WAYS = [(8, 5003, 4096, 128), (8, 4115, 8192, 64), (5, 9001, 8192, 128), (8, 33003, 8224, 256), (7, 4801, 16384, 32),
        (3, 4115, 28704, 128), (1, 4115, 5152, 64), (2, 4200, 800, 32), (4, 4099, 1024, 128), (6, 16500, 1024, 64),
        (1, 12345, 1088, 32), (2, 32771, 640, 128), (5, 32763, 4128, 128), (8, 57001, 1312, 32)]


@pytest.mark.parametrize("batch,out,inf,group", WAYS)
def test_ways(batch, out, inf, group):
    announce(f"i4group way of {batch}x{out}x{inf} group {group}")
    rng = case_rng(13, out, inf)
    m = i4_matrix(rng, out, inf, group)
    x, bias = rng.standard_normal((batch, inf)).astype(np.float32), rng.standard_normal(out).astype(np.float32)
    y = run(m, out, inf, group, x, bias)
    for rows in np.array_split(np.arange(out), -(-out * inf // (1 << 24))):
        w = i4_weights(*(v[rows] for v in m), inf, group)
        exact = x.astype(np.float64) @ w.T
        tol = i4_tolerance(w, x.astype(np.float64)) + 2.0 ** -23 * np.abs(bias[rows])
        exact = exact + bias[rows].astype(np.float64)
        err = np.abs(y[:, rows] - exact)
        assert np.all(err <= tol + 2.0 ** -24 * np.abs(exact)), (float((err / tol).max()), int(rows[np.argmax(err / tol) % len(rows)]))


@pytest.mark.parametrize("batch,out,inf,group", [(8, 4115, 4096, 128), (6, 2500, 8192, 64), (4, 9003, 8192, 32), (2, 12000, 1056, 64),
                                                 (4, 17001, 896, 128), (5, 16400, 6176, 128), (8, 32760, 2080, 64), (3, 32755, 2592, 128)])
def test_ways_of_swiglu(batch, out, inf, group):
    announce(f"i4group swiglu way of {batch}x{out}x{inf} group {group}")
    import torch
    rng = case_rng(14, out, inf)
    gate, up = (i4_matrix(rng, out, inf, group) for _ in range(2))
    x = rng.standard_normal((batch, inf)).astype(np.float32)
    buf, h = guarded_y(batch * out)
    dmv.pesti_gemv_i4group_swiglu(out, inf, group, *put(gate), *put(up), to_dev(x), h, batch)
    torch.cuda.synchronize()
    assert guards_intact(buf, batch * out)
    h, x = h.cpu().numpy().reshape(batch, out).astype(np.float64), x.astype(np.float64)
    for rows in np.array_split(np.arange(out), -(-out * inf // (1 << 24))):
        wg, wu = (i4_weights(*(v[rows] for v in m), inf, group) for m in (gate, up))
        g, u, eg, eu = x @ wg.T, x @ wu.T, i4_tolerance(wg, x), i4_tolerance(wu, x)
        tol = 1.1 * eg * (np.abs(u) + eu) + np.abs(silu(g)) * eu + 2.0 ** -20 * np.abs(silu(g) * u) + 1e-30
        err = np.abs(h[:, rows] - silu(g) * u)
        assert np.all(err <= tol), float((err / tol).max())


def test_a_group_of_all_ways():
    """Ops that are dealt out differently share a call, and keep the bits of their single calls."""
    announce("i4group group of all ways")
    import torch
    rng = case_rng(15)
    ops, singles = [], []
    for out, inf in ((4115, 8192), (40, 8192), (4800, 896), (17000, 896), (600, 4096), (9000, 8192), (3, 32)):
        p, s, z = put(i4_matrix(rng, out, inf, 128))
        x = to_dev(rng.standard_normal((8, inf)).astype(np.float32))
        y, y1 = (torch.full((8, out), 7.0, device="cuda") for _ in range(2))
        ops.append((out, inf, p, s, z, x, y, None))
        dmv.pesti_gemv_i4group(out, inf, 128, p, s, z, x, y1, None, 8)
        singles.append(y1)
    dmv.pesti_gemv_group_i4group(ops, 128, 8)
    torch.cuda.synchronize()
    for op, y1 in zip(ops, singles):
        assert torch.equal(op[6], y1), op[:2]


# large enough for the matrix cores: a wavefront a tile, dealt out, in phases, rows of less than a chunk
LARGE = [(5, 4801, 800, 32), (5, 2101, 2080, 64), (8, 1045, 8224, 128), (8, 50003, 64, 32), (7, 60005, 32, 64)]


@pytest.mark.parametrize("batch,out,inf,group", LARGE)
@pytest.mark.parametrize("size", [1e-38, 1e-20, 1.0, 3e4, 1e30])
def test_magnitudes_on_the_matrix_cores(batch, out, inf, group, size):
    announce(f"i4group {batch}x{out}x{inf} x of {size}")
    rng = case_rng(16, out)
    x = (rng.standard_normal((batch, inf)) * size).astype(np.float32)
    x[1] *= 1e-6   # columns of their own sizes
    x[2, :32] *= 1e4
    check(i4_matrix(rng, out, inf, group), out, inf, group, x)


@pytest.mark.parametrize("batch,out,inf,group", LARGE)
def test_values_on_the_matrix_cores(batch, out, inf, group):
    """Zero points of any value, scales of every kind, a row of zero weights, an element 2^27 times the others on a zero
    weight, infinities and NaN in columns of their own."""
    announce(f"i4group {batch}x{out}x{inf} values")
    rng = case_rng(17, out)
    packed, scales, zeros = m = i4_matrix(rng, out, inf, group)
    zeros[:50] = rng.integers(0, 256, zeros[:50].shape, dtype=np.uint8)
    scales[60], scales[61], scales[62], scales[63] = 0, -0.5, 6e-8, 65504
    packed[70:90], zeros[70:90] = 0x99, 9
    packed[:, 8], zeros[100:, 0] = (packed[:, 8] & 0xF0) | 7, 7   # weight 16 of rows from 100 on
    x = rng.standard_normal((batch, inf)).astype(np.float32)
    x[1, 16] = 2.0 ** 27
    x[2, 21], x[3, 5], x[3, 6], x[4, 30] = np.inf, np.inf, -np.inf, np.nan
    bias = rng.standard_normal(out).astype(np.float32)
    y = run(m, out, inf, group, x, bias)
    w = i4_weights(*m, inf, group)
    none = (w == 0).all(1)
    assert none[60] and np.array_equal(y[:2, none].astype(np.float32), np.broadcast_to(bias[none], (2, none.sum())))
    fine = [b for b in range(batch) if b not in (2, 3, 4)]
    xs = x[fine].astype(np.float64)
    exact, tol = xs @ w.T, i4_tolerance(w, xs) + 2.0 ** -23 * np.abs(bias)
    exact = exact + bias.astype(np.float64)
    err = np.abs(y[fine] - exact)
    assert np.all(err <= tol + 2.0 ** -24 * np.abs(exact)), float((err / tol).max())
    # an infinity times a weight is one of the weight's sign, times a zero weight NaN
    hit = w[:, 21]
    assert np.all(y[2][hit > 0] == np.inf) and np.all(y[2][hit < 0] == -np.inf) and np.isnan(y[2][hit == 0]).all()
    one, two = w[:, 5], w[:, 6]
    assert np.isnan(y[3][one * two >= 0]).all() and np.all(y[3][(one > 0) & (two < 0)] == np.inf)
    assert np.isnan(y[4]).all()


@pytest.mark.parametrize("batch,out,inf,group", LARGE)
def test_surroundings_on_the_matrix_cores(batch, out, inf, group):
    announce(f"i4group {batch}x{out}x{inf} surroundings")
    import torch
    rng = case_rng(18, out)
    m = i4_matrix(rng, out, inf, group)
    x = to_dev(rng.standard_normal((batch, inf)).astype(np.float32))
    ys = []
    for fill in (0, 255):
        dev = []
        for a in m:
            a = np.ascontiguousarray(a)
            whole = torch.full((a.nbytes + 512,), fill, dtype=torch.uint8, device="cuda")
            whole[256:256 + a.nbytes] = torch.from_numpy(a.reshape(-1).view(np.uint8)).cuda()
            dev.append(whole[256:256 + a.nbytes])
        buf, y = guarded_y(batch * out)
        dmv.pesti_gemv_i4group(out, inf, group, dev[0], dev[1].view(torch.float16), dev[2], x, y, None, batch)
        torch.cuda.synchronize()
        assert guards_intact(buf, batch * out)
        ys.append(y.cpu())
    assert torch.equal(*ys)
