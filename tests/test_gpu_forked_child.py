"""A child forked after the GPU was used is refused by torch's own error, as before the compiled checks; the parent goes on."""
from __future__ import annotations

import os

import pytest

import dequantize_mat_vec_amd as dmv
from dequantize_mat_vec_amd import _lib
from gpu_util import announce
from test_gpu_fast_calls import fixture

pytestmark = pytest.mark.gpu


def answer_of_a_child(call):
    """What call() raises in a forked child (which does nothing else and ends at once)."""
    read, write = os.pipe()
    pid = os.fork()
    if pid == 0:
        try:
            try:
                text = f"returned {call()!r}"
            except BaseException as e:
                text = f"{type(e).__name__}: {e}"
            os.write(write, text[:2000].encode())
        finally:
            os._exit(0)
    os.close(write)
    with os.fdopen(read) as f:
        text = f.read()
    assert os.waitpid(pid, 0)[1] == 0
    return text


def test_a_forked_child_is_refused():
    announce("forked child")
    import torch
    _, free = fixture()["pesti_cache_free"]
    assert dmv.pesti_cache_free(**free) == 0
    assert _lib._place(None)[1] == torch.cuda.current_device()
    # neither would reach the GPU in the child: the one looks up the device, the other has an empty list
    for call in (lambda: _lib._place(None), lambda: dmv.pesti_cache_free(free["cache"], free["table"], 0)):
        text = answer_of_a_child(call)
        assert text.startswith("RuntimeError: ") and "fork" in text, text
    assert dmv.pesti_cache_free(**free) == 0
    torch.cuda.synchronize()
