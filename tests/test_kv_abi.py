"""Refusals of the 4-bit mat-vec with group scales and of the paged cache's
calls, before any device work (safe without a GPU: nothing is launched), the
binding's own checks, and the plain forms that the GPU tests compare with."""
from __future__ import annotations

import ctypes
import re
from pathlib import Path

import numpy as np
import pytest

import dequantize_mat_vec_amd as dmv
import kv_reference as ref
from dequantize_mat_vec_amd import _lib
from test_experts_types import DeviceTensor

HEADER = Path(__file__).resolve().parent.parent / "include" / "pesti.h"
FAKE = 0x100000   # 16-byte aligned, never dereferenced (calls are rejected)
F16, F32, I8, Q8 = 16, 17, 3, 0
SHAPE, NULL, BATCH, ALIGN, WORKSPACE = (_lib.PESTI_ERR_SHAPE, _lib.PESTI_ERR_NULL, _lib.PESTI_ERR_BATCH, _lib.PESTI_ERR_ALIGN,
                                        _lib.PESTI_ERR_WORKSPACE)


def lib():
    return _lib.load()


def addr(s):
    return None if s is None else ctypes.addressof(s)


def test_constants_match_the_header():
    text = HEADER.read_text()
    for name, fid in dmv.CACHE_FORMAT_IDS.items():
        assert re.search(rf"#define PESTI_FMT_{name.upper()} {fid}\b", text), name


# --- 4-bit weights with group scales ------------------------------------------
def test_i4group_refusals():
    f = lib().pesti_gemv_i4group

    def call(out=8, inf=64, group=32, p=FAKE, s=FAKE, z=None, x=FAKE, y=FAKE, b=None, batch=1):
        return f(out, inf, group, p, s, z, x, y, b, batch, None)

    for group in (0, -32, 16, 31, 33, 48, 96, 65536, 1 << 40):
        assert call(group=group) == SHAPE, group
    for inf in (-32, 40, 16, 32800):
        assert call(inf=inf) == SHAPE, inf
    assert call(out=-1) == SHAPE and call(out=1 << 31) == SHAPE
    assert call(batch=-1) == BATCH and call(batch=9) == BATCH
    for name in ("p", "s", "x", "y"):
        assert call(**{name: None}) == NULL, name
    for name in ("p", "x", "y"):
        assert call(**{name: FAKE + 8}) == ALIGN, name
    assert call(s=FAKE + 1) == ALIGN and call(b=FAKE + 2) == ALIGN
    assert call(out=0, p=None, s=None, x=None, y=None) == 0
    assert call(batch=0, p=None, s=None, x=None, y=None) == 0


def test_i4group_grouped_refusals():
    f = lib().pesti_gemv_group_i4group

    def op(out=8, inf=64, p=FAKE, s=FAKE, z=None, x=FAKE, y=FAKE, b=None):
        return dmv.GemvI4GroupOp(out, inf, p, s, z, x, y, b)

    def call(*ops, n=None, group=32, batch=1):
        arr = (dmv.GemvI4GroupOp * max(len(ops), 1))(*ops)
        return f(len(ops) if n is None else n, ctypes.cast(arr, ctypes.c_void_p), group, batch, None)

    assert f(2, None, 32, 1, None) == NULL and f(0, None, 32, 1, None) == 0
    assert call(op(), n=-1) == SHAPE and call(op(), n=9) == SHAPE
    assert call(op(), group=48) == SHAPE and call(op(), batch=9) == BATCH
    assert call(op(), op(inf=40)) == SHAPE and call(op(), op(y=None)) == NULL and call(op(), op(x=FAKE + 4)) == ALIGN
    assert call(op(out=0), op(out=0, y=None)) == 0


def test_i4group_swiglu_and_dequant_refusals():
    f = lib().pesti_gemv_i4group_swiglu

    def call(out=8, inf=64, group=64, gp=FAKE, gs=FAKE, up=FAKE, us=FAKE, x=FAKE, h=FAKE, batch=1):
        return f(out, inf, group, gp, gs, None, up, us, None, x, h, batch, None)

    assert call(group=100) == SHAPE and call(inf=48) == SHAPE and call(out=-1) == SHAPE and call(batch=9) == BATCH
    for name in ("gp", "gs", "up", "us", "x", "h"):
        assert call(**{name: None}) == NULL, name
    for name in ("gp", "up", "x", "h"):
        assert call(**{name: FAKE + 8}) == ALIGN, name
    assert call(us=FAKE + 1) == ALIGN and call(out=0, h=None) == 0 and call(batch=0, h=None) == 0
    d = lib().pesti_dequant_i4group
    assert d(4, 64, 31, FAKE, FAKE, None, FAKE, None) == SHAPE
    assert d(-1, 64, 32, FAKE, FAKE, None, FAKE, None) == SHAPE
    assert d(4, 72, 32, FAKE, FAKE, None, FAKE, None) == SHAPE
    assert d(4, 64, 32, None, FAKE, None, FAKE, None) == NULL
    assert d(4, 64, 32, FAKE, None, None, FAKE, None) == NULL
    assert d(4, 64, 32, FAKE, FAKE, None, None, None) == NULL
    assert d(4, 64, 32, FAKE, FAKE, None, FAKE + 4, None) == ALIGN
    assert d(0, 64, 32, None, None, None, None, None) == 0


# --- cache ------------------------------------------------------------------------
def cache(**kw):
    a = dict(format=F16, layers=2, pages=8, page_size=16, kv_heads=2, head_dim=64, k=FAKE, v=FAKE, k_scales=None, v_scales=None)
    a.update(kw)
    return dmv.KvCache(*(a[n] for n, _ in dmv.KvCache._fields_))


def table(**kw):
    a = dict(seqs=4, width=3, table=FAKE, lengths=FAKE, refs=FAKE)
    a.update(kw)
    return dmv.KvTable(*(a[n] for n, _ in dmv.KvTable._fields_))


def extend(c, t, n=2, ids=FAKE, counts=FAKE, status=FAKE):
    return lib().pesti_cache_extend(addr(c), addr(t), n, ids, counts, status, None)


def append(c, t, layer=0, rows=2, fmt=F16, k=FAKE, v=FAKE, stride=128, ids=FAKE, pos=FAKE):
    return lib().pesti_cache_append(addr(c), addr(t), layer, rows, fmt, k, v, stride, ids, pos, None)


def attend(c, t, layer=0, rows=2, heads=4, ids=FAKE, qf=F32, q=FAKE, stride=256, yf=F32, y=FAKE, most=48, ws=FAKE, ws_bytes=1 << 30):
    return lib().pesti_attn_paged(addr(c), addr(t), layer, rows, heads, ids, qf, q, stride, yf, y, 1.0, most, ws, ws_bytes, None)


def fork(c, t, n=2, parents=FAKE, children=FAKE, status=FAKE, ws=FAKE, ws_bytes=1 << 20):
    return lib().pesti_cache_fork(addr(c), addr(t), n, parents, children, status, ws, ws_bytes, None)


def free(c, t, n=2, ids=FAKE):
    return lib().pesti_cache_free(addr(c), addr(t), n, ids, None)


def compact(c, t, live=FAKE, ws=FAKE, ws_bytes=1 << 20):
    return lib().pesti_cache_compact(addr(c), addr(t), live, ws, ws_bytes, None)


def copy(c, _t, n=2, src=FAKE, dst=FAKE):
    return lib().pesti_cache_copy_pages(addr(c), n, src, dst, None)


CALLS = [extend, append, attend, fork, free, compact, copy]
BAD_SIZES = [dict(format=Q8), dict(format=F32), dict(layers=0), dict(layers=1025), dict(pages=-1), dict(pages=(1 << 22) + 1),
             dict(page_size=4), dict(page_size=24), dict(page_size=2048), dict(page_size=0), dict(page_size=-16), dict(kv_heads=0),
             dict(kv_heads=1025), dict(head_dim=0), dict(head_dim=48), dict(head_dim=288), dict(head_dim=-32)]


@pytest.mark.parametrize("call", CALLS)
def test_cache_sizes_are_refused(call):
    for bad in BAD_SIZES:
        assert call(cache(**bad), table()) == SHAPE, bad
    assert call(None, table()) == NULL
    if call is not copy:
        assert call(cache(), None) == NULL
        for bad in (dict(seqs=-1), dict(seqs=4097), dict(width=-1), dict(width=(1 << 26) + 1)):
            assert call(cache(), table(**bad)) == SHAPE, bad


@pytest.mark.parametrize("call", CALLS)
def test_missing_and_unaligned_arrays_are_refused(call):
    if call is not copy:
        assert call(cache(), table(lengths=None)) == NULL and call(cache(), table(table=None)) == NULL
        assert call(cache(), table(lengths=FAKE + 2)) == ALIGN and call(cache(), table(table=FAKE + 1)) == ALIGN
    if call in (extend, fork, free, compact):
        assert call(cache(), table(refs=None)) == NULL and call(cache(), table(refs=FAKE + 2)) == ALIGN
    if call in (append, attend, fork, compact, copy):
        i8 = dict(format=I8, k_scales=FAKE, v_scales=FAKE)
        for name in ("k", "v"):
            assert call(cache(**{name: None}), table()) == NULL and call(cache(**{name: FAKE + 8}), table()) == ALIGN
        for name in ("k_scales", "v_scales"):
            assert call(cache(**{**i8, name: None}), table()) == NULL
            assert call(cache(**{**i8, name: FAKE + 8}), table()) == ALIGN


@pytest.mark.parametrize("call", [extend, fork, free])
def test_list_lengths(call):
    assert call(cache(), table(), n=-1) == BATCH and call(cache(), table(seqs=4096), n=4097) == BATCH
    assert call(cache(), table(), n=0) == 0


def test_lists():
    c, t = cache(), table()
    assert extend(c, t, status=None) == NULL
    for name in ("ids", "counts", "status"):
        assert extend(c, t, **{name: FAKE + 2}) == ALIGN, name
    for name in ("parents", "children", "status"):
        assert fork(c, t, **{name: None}) == NULL and fork(c, t, **{name: FAKE + 1}) == ALIGN, name
    assert fork(c, t, n=5) == BATCH
    assert free(c, t, ids=FAKE + 2) == ALIGN
    assert compact(c, t, live=None) == NULL and compact(c, t, live=FAKE + 2) == ALIGN
    assert copy(c, t, n=-1) == BATCH and copy(c, t, n=(1 << 22) + 1) == BATCH and copy(c, t, n=0, src=None) == 0
    for name in ("src", "dst"):
        assert copy(c, t, **{name: None}) == NULL and copy(c, t, **{name: FAKE + 2}) == ALIGN, name


def test_cache_workspace():
    c, t = cache(), table()
    need = lib().pesti_cache_workspace_bytes(addr(c), addr(t))
    assert need > 0
    for call in (fork, compact):
        assert call(c, t, ws=None) == WORKSPACE and call(c, t, ws_bytes=need - 1) == WORKSPACE and call(c, t, ws_bytes=-1) == WORKSPACE
        assert call(c, t, ws=FAKE + 8) == ALIGN
    assert lib().pesti_cache_workspace_bytes(addr(cache(page_size=9)), addr(t)) == SHAPE
    assert lib().pesti_cache_workspace_bytes(addr(c), addr(table(seqs=-1))) == SHAPE
    assert lib().pesti_cache_workspace_bytes(None, addr(t)) == NULL and lib().pesti_cache_workspace_bytes(addr(c), None) == NULL


def test_append_refusals():
    c, t = cache(), table()
    assert append(c, t, layer=-1) == SHAPE and append(c, t, layer=2) == SHAPE
    assert append(c, t, fmt=I8) == SHAPE and append(c, t, stride=127) == SHAPE and append(c, t, stride=1 << 41) == SHAPE
    assert append(c, t, rows=-1) == BATCH and append(c, t, rows=(1 << 20) + 1) == BATCH
    for name in ("k", "v"):
        assert append(c, t, **{name: None}) == NULL and append(c, t, **{name: FAKE + 8}) == ALIGN, name
    assert append(c, t, stride=132) == ALIGN and append(c, t, fmt=F32, stride=130) == ALIGN
    assert append(c, t, ids=FAKE + 2) == ALIGN and append(c, t, pos=FAKE + 2) == ALIGN
    assert append(c, t, rows=0, k=None, v=None) == 0


def test_attention_refusals():
    c, t = cache(), table()
    assert attend(c, t, layer=-1) == SHAPE and attend(c, t, layer=2) == SHAPE
    for heads in (0, -2, 3, 1026):
        assert attend(c, t, heads=heads, stride=1 << 20) == SHAPE, heads
    assert attend(c, t, qf=I8) == SHAPE and attend(c, t, yf=Q8) == SHAPE
    assert attend(c, t, stride=255) == SHAPE and attend(c, t, stride=1 << 41) == SHAPE
    assert attend(c, t, most=0) == SHAPE and attend(c, t, most=(1 << 30) + 1) == SHAPE
    assert attend(c, t, rows=-1) == BATCH and attend(c, t, rows=4097) == BATCH
    for name in ("q", "y"):
        assert attend(c, t, **{name: None}) == NULL and attend(c, t, **{name: FAKE + 8}) == ALIGN, name
    assert attend(c, t, stride=258) == ALIGN and attend(c, t, qf=F16, stride=260) == ALIGN and attend(c, t, ids=FAKE + 2) == ALIGN
    assert attend(c, t, rows=0, q=None, y=None) == 0


def test_attention_workspace():
    f = lib().pesti_attn_paged_workspace_bytes
    c = cache()
    assert f(addr(c), 1, 4, 0) == SHAPE and f(addr(c), 1, 3, 9) == SHAPE and f(addr(c), -1, 4, 9) == BATCH and f(None, 1, 4, 9) == NULL
    assert f(addr(cache(head_dim=33)), 1, 4, 9) == SHAPE
    sizes = [f(addr(c), 1, 4, n) for n in (1, 100, 10000, 1 << 20, 1 << 30)]
    assert all(s >= 0 for s in sizes) and sizes == sorted(sizes) and sizes[-1] <= 1 << 30
    assert f(addr(c), 4096, 1024, 1 << 30) >= 0
    need = f(addr(c), 1, 4, 1 << 20)
    if need:
        assert attend(c, table(), rows=1, most=1 << 20, ws=None) == WORKSPACE
        assert attend(c, table(), rows=1, most=1 << 20, ws_bytes=need - 1) == WORKSPACE
        assert attend(c, table(), rows=1, most=1 << 20, ws=FAKE + 4) == ALIGN


# --- binding ------------------------------------------------------------------------
class Rows(DeviceTensor):
    """What the binding asks of a two-dimensional tensor whose rows may lie apart."""

    def __init__(self, dtype, rows, width, apart=None, held=None):
        super().__init__(dtype, rows * width)
        self.shape, self.apart = (rows, width), apart or width
        self.held = (held or (rows - 1) * self.apart + width) * dtype.itemsize

    def stride(self):
        return self.apart, 1

    def storage_offset(self):
        return 0

    def untyped_storage(self):
        return type("Storage", (), {"nbytes": lambda _s: self.held})()


class Apart(Rows):
    def stride(self):
        return 256, 2


def test_binding_checks_sizes_and_types():
    import torch
    f16, f32, i8, i32, u8 = torch.float16, torch.float32, torch.int8, torch.int32, torch.uint8
    t = DeviceTensor
    good = dict(packed=t(u8, 8 * 20), scales=t(f16, 8 * 2), zeros=t(u8, 16), x=t(f32, 40), y=t(f32, 8), bias=t(f32, 8))

    def gemv(**kw):   # 40 columns: refused by the library, so nothing is launched
        a = {**good, **kw}
        return dmv.pesti_gemv_i4group(8, 40, 32, a["packed"], a["scales"], a["zeros"], a["x"], a["y"], a["bias"], stream=0)

    with pytest.raises(dmv.PestiError):
        gemv()
    for name, bad in (("packed", t(i8, 160)), ("packed", t(u8, 159)), ("scales", t(torch.bfloat16, 16)), ("scales", t(f16, 15)),
                      ("zeros", t(i8, 16)), ("zeros", t(u8, 15)), ("x", t(f16, 80)), ("y", t(f32, 7)), ("bias", t(f16, 16))):
        with pytest.raises(ValueError, match=name):
            gemv(**{name: bad})
    ops = dmv.gemv_i4group_ops([(8, 40, *(good[n] for n in ("packed", "scales", "zeros", "x", "y", "bias")))], 32, 1)
    with pytest.raises(dmv.PestiError):
        dmv.pesti_gemv_group_i4group(ops, 32, 1, stream=0)
    for group, batch in ((64, 1), (32, 2)):
        with pytest.raises(ValueError, match="built for"):
            dmv.pesti_gemv_group_i4group(ops, group, batch, stream=0)
    rows = 2 * 8 * 2 * 16
    with pytest.raises(ValueError, match="k "):
        dmv.kv_cache("f16", 2, 8, 16, 2, 64, t(f16, rows * 64 - 1), t(f16, rows * 64))
    with pytest.raises(ValueError, match="v must"):
        dmv.kv_cache("f16", 2, 8, 16, 2, 64, t(f16, rows * 64), t(torch.bfloat16, rows * 64))
    with pytest.raises(ValueError, match="k_scales"):
        dmv.kv_cache("i8row", 2, 8, 16, 2, 64, t(i8, rows * 64), t(i8, rows * 64), t(f32, rows - 1), t(f32, rows))
    for name, bad in (("table", (t(i32, 11), t(i32, 4), t(i32, 8))), ("lengths", (t(i32, 12), t(torch.int64, 4), t(i32, 8))),
                      ("refs", (t(i32, 12), t(i32, 4), t(f32, 8)))):
        with pytest.raises(ValueError, match=name):
            dmv.kv_table(*bad, seqs=4, width=3)


def test_binding_checks_cache_calls():
    import torch
    f16, f32, i32 = torch.float16, torch.float32, torch.int32
    t = DeviceTensor
    rows = 2 * 8 * 2 * 16
    c = dmv.kv_cache("f16", 2, 8, 16, 2, 64, t(f16, rows * 64), t(f16, rows * 64))
    refs = t(i32, 7)
    refs.numel = lambda: 7
    short = dmv.kv_table(t(i32, 12), t(i32, 4), refs, 4, 3)
    with pytest.raises(ValueError, match="refs holds 7 pages"):
        dmv.pesti_cache_free(c, short, 2, None, stream=0)
    tab = dmv.kv_table(t(i32, 12), t(i32, 4), None, 4, 3)
    with pytest.raises(dmv.PestiError):   # layer 2 of two: refused by the library
        dmv.pesti_cache_append(c, tab, 2, 3, Rows(f16, 3, 128, 400), Rows(f16, 3, 128, 400), stream=0)
    for k, v, what in ((Rows(f16, 3, 128, 400), Rows(f16, 3, 128, 408), "one row stride"), (Rows(f16, 2, 128), Rows(f16, 3, 128), "k: 3 rows"),
                       (Rows(f16, 3, 128), Rows(f32, 3, 128), "v must"), (Rows(f16, 3, 128), Rows(f16, 3, 128, held=383), "v: 3 rows"), (Apart(f16, 3, 128), Rows(f16, 3, 128), "contiguous")):
        with pytest.raises(ValueError, match=what):
            dmv.pesti_cache_append(c, tab, 2, 3, k, v, stream=0)
    with pytest.raises(ValueError, match="positions"):
        dmv.pesti_cache_append(c, tab, 2, 3, Rows(f16, 3, 128), Rows(f16, 3, 128), positions=t(i32, 2), stream=0)
    for kw, what in ((dict(q=Rows(f32, 1, 256)), "q: 2 rows"), (dict(y=t(f32, 511)), "y holds"), (dict(seq_ids=t(i32, 1)), "seq_ids"),
                     (dict(q=Rows(torch.bfloat16, 2, 256)), "q: give"), (dict(workspace=t(torch.uint8, 8), workspace_bytes=9), "workspace")):
        a = dict(q=Rows(f32, 2, 256), y=t(f32, 512), **{k: v for k, v in kw.items() if k not in ("q", "y")})
        a.update({k: v for k, v in kw.items() if k in ("q", "y")})
        q, y = a.pop("q"), a.pop("y")
        a.setdefault("workspace_bytes", 0)
        with pytest.raises(ValueError, match=what):
            dmv.pesti_attn_paged(c, tab, 2, 2, 4, q, y, 1.0, stream=0, **a)


# --- the plain forms -----------------------------------------------------------------
def test_plain_codes_are_the_exact_quotients():
    from fractions import Fraction
    rng = np.random.default_rng(5)
    x = (rng.standard_normal((40, 32)) * np.exp(5 * rng.standard_normal((40, 1)))).astype(np.float32)
    x[0, :4] = 127, 0.5, 1.5, -2.5
    x[1] = 0
    codes, scales = ref.i8_rows(x.astype(np.float64))
    for row, c, s in zip(x, codes, scales):
        assert s == np.float32(np.abs(row).max() / np.float32(127))
        for v, q in zip(row, c):
            if s == 0:
                assert q == 0
                continue
            ratio = abs(Fraction(float(v)) / Fraction(float(s)))
            whole = int(ratio + Fraction(1, 2))
            assert abs(int(q)) == min(whole, 127) and (q == 0 or (q > 0) == (v > 0))


def test_plain_upkeep_keeps_its_counts():
    """Random calls: refs count the table's entries, sequences share only whole pages, and contents stay with their tokens."""
    rng = np.random.default_rng(6)
    c = ref.Cache(rng, "f16", 1, 50, 8, 1, 32, 8, 6, [])
    told = {}
    for _ in range(400):
        kind = rng.integers(0, 4)
        seqs = [int(s) for s in rng.integers(0, 8, rng.integers(1, 4))]
        if kind == 0:
            before = c.lengths.copy()
            c.extend(seqs, rng.integers(0, 12, len(seqs)))
            for s in set(seqs):
                for t in range(before[s], c.lengths[s]):
                    x = rng.standard_normal((1, 1, 32)).astype(np.float16)
                    c.append(0, x, x, [s], [t])
                    told.setdefault(s, []).append(x[0, 0])
        elif kind == 1:
            c.free(seqs)
            for s in seqs:
                told.pop(s, None)
        elif kind == 2:
            parents = [int(s) for s in rng.integers(0, 8, len(seqs))]
            empty = {s: c.length(s) == 0 for s in range(8)}
            old = {s: list(v) for s, v in told.items()}
            if c.fork(parents, seqs) == 0:
                done = set()
                for p, s in zip(parents, seqs):
                    if empty[s] and s not in done and old.get(p):
                        told[s] = list(old[p])
                    done.add(s)
        else:
            c.compact()
        held = [c.table[s, j] for s in range(8) for j in range(c.held(s))]
        assert np.array_equal(np.bincount(held, minlength=50) if held else np.zeros(50), c.refs)
        for s in range(8):
            k, there = c.rows("k", 0, s, 0)
            assert there.all() and len(k) == len(told.get(s, []))
            if len(k):
                assert np.array_equal(k, np.array(told[s], np.float64))
