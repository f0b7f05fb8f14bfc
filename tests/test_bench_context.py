"""Host logic of the decode step with a cache, of the suite's 4-bit cases and of the oracle's forms for both (no GPU)."""
from __future__ import annotations

import os
import sys

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import bench  # noqa: E402
import oracle  # noqa: E402
from dequantize_mat_vec_amd import synth  # noqa: E402
from kv_reference import Cache, i4_weights, i8_rows  # noqa: E402


def test_the_default_step_has_no_cache():
    a = bench.parse_args([])
    assert a.context is None and a.cache_format == "f16"


def test_bytes_of_the_context():
    assert bench.context_bytes(1000, "f16") == 24 * 2 * 1000 * 2 * 64 * 2
    assert bench.context_bytes(1000, "i8row") == 24 * 2 * 1000 * 2 * (64 + 4)
    assert bench.context_bytes(0, "f16") == 0


def test_the_earlier_suite_cases_keep_their_places():
    cases = bench.suite_cases()
    first = next(i for i, c in enumerate(cases) if c[1] == "gemv4")
    assert all(c[1] == "gemv4" for c in cases[first:]) and len(cases) - first == 6
    assert all(c[1] != "gemv4" for c in cases[:first])
    assert len({c[0] for c in cases}) == len(cases)


def test_suite_inputs_of_a_4_bit_case():
    i, (name, kind, prm) = [(i, c) for i, c in enumerate(bench.suite_cases()) if c[1] == "gemv4"][-1]
    d = bench.suite_case_inputs(i, name, kind, prm, 40)
    assert d["codes"].shape == (40, 2432) and d["scales"].shape == d["zeros"].shape == (40, 38)
    assert d["packed"].size == 40 * (2432 + 3 * 38)
    assert np.array_equal(d["packed"][40 * 2432:40 * 2432 + 80 * 38].view(np.float16), d["scales"].reshape(-1))
    assert d["algo"] == 40 * (2432 + 3 * 38) + 4 * (4864 + 40)


@pytest.mark.parametrize("rows,inf,group,zeros", [(3, 64, 32, True), (5, 96, 64, True), (2, 32, 128, False)])
def test_oracle_of_4_bit_weights(rows, inf, group, zeros):
    rng = np.random.default_rng([rows, inf])
    packed, scales, z = synth.i4group(rng, rows, inf, group)
    z = z if zeros else None
    w = oracle.dequant_i4group(packed, rows, inf, group, scales, z)
    assert np.array_equal(w, i4_weights(packed, scales, z, inf, group))
    x, b = synth.activations(rng, 2, inf), synth.bias(rng, rows)
    y, size = oracle.gemv_i4group(packed, rows, inf, group, scales, z, x, b, row_chunk=2)
    assert np.allclose(y, x.astype(np.float64) @ w.T + b, rtol=1e-12) and (size >= np.abs(y) * (1 - 1e-12)).all()


@pytest.mark.parametrize("fmt", ("f16", "i8row"))
def test_oracle_of_attention(fmt):
    rng = np.random.default_rng(5)
    c = Cache(rng, fmt, 2, 9, 8, 2, 32, 2, 5, (33, 7))
    q = rng.standard_normal((2, 4, 32))
    want, _ = c.attend(1, q, 0.2)
    for s, h in np.ndindex(2, 4):
        k, v = (oracle.cached_rows(getattr(c, n)[1], None if fmt == "f16" else getattr(c, n + "_scales")[1], c.table[s],
                                   int(c.lengths[s]), h // 2) for n in ("k", "v"))
        y, size = oracle.attend(q[s, h], k, v, 0.2)
        assert np.allclose(y, want[s, h], rtol=0, atol=1e-13) and (size >= np.abs(y) - 1e-15).all()


def test_oracle_of_attention_over_nothing():
    y, size = oracle.attend(np.ones(32), np.zeros((0, 32)), np.zeros((0, 32)), 1.0)
    assert not y.any() and not size.any()


def cached_sample(fmt):
    """What StepCache.sample gives after a step, from host values alone."""
    rng = np.random.default_rng(7)
    length, pages, d, kvh = 150, 3, synth.QWEN_HEAD_DIM, synth.QWEN_KV_HEADS
    c = Cache(rng, fmt, 1, pages, bench.CACHE_PAGE_SIZE, kvh, d, 1, pages, (length,))
    q = rng.standard_normal((synth.QWEN_HEADS, d)).astype(np.float32)
    k, v = (rng.standard_normal((1, kvh, d)).astype(np.float32) for _ in range(2))
    c.append(0, k, v, [0], [length - 1])
    y, _ = c.attend(0, q[None], d ** -0.5)
    out = {"cache_layers": [0], "cache_length": length, "cache_status": 0, "cache_table": c.table[0], "cache_q_0": q.reshape(-1),
           "cache_k_0": k.reshape(-1), "cache_v_0": v.reshape(-1), "cache_y_0": y[0].astype(np.float32).reshape(-1),
           "cache_k_pool_0": c.k[0], "cache_v_pool_0": c.v[0]}
    if fmt == "i8row":
        out.update(cache_k_scales_0=c.k_scales[0], cache_v_scales_0=c.v_scales[0])
    return out


@pytest.mark.parametrize("fmt", ("f16", "i8row"))
def test_cache_parity_accepts_the_plain_result_and_names_planted_errors(fmt):
    n, bad, worst = bench.cache_parity(cached_sample(fmt))
    assert n == 14 * 64 and not bad and worst < 1.0
    s = cached_sample(fmt)
    s["cache_y_0"][9 * 64 + 3] += 0.01                     # one value of head 9
    assert bench.cache_parity(s)[1] == ["attention: layer 0, head 9"]
    s = cached_sample(fmt)
    s["cache_v_0"][64 + 5] += 1.0                          # what the V call wrote is not what the cache holds
    assert any("KV head 1: the step's V" in f for f in bench.cache_parity(s)[1])
    s = cached_sample(fmt)
    s["cache_status"] = 1                                  # pages were missing
    assert bench.cache_parity(s)[1]


def test_reference_rounding_agrees_with_the_oracle():
    x = np.random.default_rng(3).standard_normal((5, 64)).astype(np.float32)
    codes, scales = i8_rows(x)
    q, s = oracle.quantize_i8token(x)
    assert np.array_equal(codes, q) and np.array_equal(scales, s)


def test_a_context_out_of_range_is_refused(capsys):
    for n in ("-1", "1048577"):
        assert bench.main(["--context", n]) == 2
        assert "--context" in capsys.readouterr().err
