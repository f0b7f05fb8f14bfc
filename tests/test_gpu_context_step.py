"""The decode step with its cache on the GPU: eager steps and replays of a captured one, checked as the benchmark does."""
from __future__ import annotations

import os
import sys

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt,context,grouping,ffn", [("f16", 0, "stage", "separate"), ("f16", 1000, "none", "separate"),
                                                      ("i8row", 333, "stage", "swiglu"), ("f16", 9000, "stage", "separate"),
                                                      ("i8row", 70000, "stage", "separate")])
def test_step_with_a_cache(fmt, context, grouping, ffn):
    import torch
    import bench
    import dequantize_mat_vec_amd as dmv
    from dequantize_mat_vec_amd import synth
    lib = dmv.load()
    calls, weights, xs, ys, biases = bench.build_inputs(2, synth.decode_step_calls(layers=2))
    cache = bench.StepCache(lib, context, fmt, 16, calls, xs, ys)
    before = [t.clone() for t in (cache.k, cache.v)]
    step = bench.make_step(lib, calls, bench.plan_launches(calls, grouping), weights, xs, ys, biases, ffn, cache)
    stream = torch.cuda.Stream()

    def check(tokens):
        torch.cuda.synchronize()
        s = cache.sample((0, 1), calls, xs, ys)
        assert s["cache_length"] == context + tokens
        n, bad, worst = bench.cache_parity(s)
        assert n == 2 * 14 * 64 and not bad and worst < 1.0

    with torch.cuda.stream(stream):
        for i in range(2):
            step(i, stream.cuda_stream)
            check(1 + i)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            step(0, torch.cuda.current_stream().cuda_stream)
        for i in range(4):
            for y in ys:
                y.fill_(float("nan"))
            graph.replay()
            check(3 + i)
        step(1, stream.cuda_stream, {"cache"})   # the cache's launches alone
        check(7)
    # tokens that were there are there still
    held = context // bench.CACHE_PAGE_SIZE
    pages = cache.pages[0, :held].long()
    for was, now in zip(before, (cache.k, cache.v)):
        assert torch.equal(was[:, pages], now[:, pages])
    # O was fed by the attention: its output is the product with the attention's result
    o = next(i for i, c in enumerate(calls) if c[1] == "o")
    import oracle
    step(0, torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    packed = bench.host_inputs([calls[o]])[0][0]
    y, size = oracle.gemv_packed(calls[o][2], packed, calls[o][3], calls[o][4], xs[o].cpu().numpy()[None])
    assert (np.abs(ys[o].cpu().numpy() - y[0]) <= 1e-4 * size[0] + 1e-6).all()


def test_a_full_table_stops_growing():
    """Past the pages that it was made for the step reports it and leaves the tokens as they are."""
    import torch
    import bench
    import dequantize_mat_vec_amd as dmv
    from dequantize_mat_vec_amd import synth
    lib = dmv.load()
    calls, weights, xs, ys, biases = bench.build_inputs(1, synth.decode_step_calls(layers=1))
    cache = bench.StepCache(lib, 63, "f16", 1, calls, xs, ys)
    step = bench.make_step(lib, calls, bench.plan_launches(calls, "stage"), weights, xs, ys, biases, "separate", cache)
    for want in ((64, 0), (64, -1)):
        step(0, torch.cuda.current_stream().cuda_stream)
        torch.cuda.synchronize()
        assert (cache.lengths.item(), cache.status.item()) == want
