"""The build and the binding where the compiled argument checks cannot be had: the library is linked all the same, what an
earlier build left is gone, and the checks in Python do alone (no GPU needed)."""
from __future__ import annotations

import ctypes
import subprocess
import sys
from pathlib import Path

import pytest

import dequantize_mat_vec_amd
from dequantize_mat_vec_amd import build

ROOT = Path(dequantize_mat_vec_amd.__file__).resolve().parent.parent


def no_torch(_out):
    raise ImportError("no torch here")


def no_compiler(_out):
    return ["/nowhere/c++"]


def no_headers(out):
    return [sys.executable, "-c", f"open({str(out)!r}, 'w').write('half'); raise SystemExit('Python.h: no such file')"]


@pytest.mark.parametrize("command", [no_torch, no_compiler, no_headers])
def test_the_library_is_linked_without_the_argument_checks(command, tmp_path, monkeypatch, capsys):
    (tmp_path / "csrc").mkdir()
    (tmp_path / "csrc" / "one.hip").write_text('extern "C" int answer() { return 42; }\n')
    stale = [tmp_path / "_tensor_args.so", tmp_path / build.ARGS_PATH.name]
    for p in stale:
        p.write_text("of an earlier build")
    for name, value in (("PKG_DIR", tmp_path), ("SRC_DIR", tmp_path / "csrc"), ("LIB_PATH", tmp_path / "lib.so"),
                        ("ARGS_PATH", stale[1]), ("args_command", command)):
        monkeypatch.setattr(build, name, value)
    assert build.build() == tmp_path / "lib.so"
    assert ctypes.CDLL(str(tmp_path / "lib.so")).answer() == 42
    assert not list(tmp_path.rglob("*tensor_args*.so*"))
    assert "left out" in capsys.readouterr().err


def test_an_error_in_a_hip_source_is_still_one(tmp_path, monkeypatch, capsys):
    (tmp_path / "csrc").mkdir()
    (tmp_path / "csrc" / "one.hip").write_text("no C++\n")
    for name, value in (("PKG_DIR", tmp_path), ("SRC_DIR", tmp_path / "csrc"), ("LIB_PATH", tmp_path / "lib.so"),
                        ("args_command", no_torch)):
        monkeypatch.setattr(build, name, value)
    with pytest.raises(RuntimeError, match="HIP compilation failed"):
        build.build()
    assert not (tmp_path / "lib.so").exists() and "one.hip" in capsys.readouterr().err


WITHOUT = """
import sys, types
sys.path[:0] = [{root!r}, {tests!r}]
import torch
import dequantize_mat_vec_amd as dmv
name = "dequantize_mat_vec_amd._tensor_args"
if {other!r}:   # checks built for another torch, or by an earlier build that did not say, that must not be asked
    sys.modules[name] = dmv._tensor_args = types.SimpleNamespace(**(dict() if {other!r} == "unsaid" else dict(torch={other!r})))
else:
    sys.modules[name] = None
from dequantize_mat_vec_amd import _lib
from test_experts_types import DeviceTensor as T
from test_kv_abi import Rows
lib = _lib.load()
assert _lib._sized.__module__ == _lib._rows.__module__ == _lib.__name__ and _lib._call_attn_paged is _lib._not_made
f32, f16, i8, i32, u8 = torch.float32, torch.float16, torch.int8, torch.int32, torch.uint8
def refused(kind, call):
    try:
        call()
    except kind as e:
        return str(e)
    raise SystemExit("no error")
refused(dmv.PestiError, lambda: dmv.pesti_gemv_i4group(8, 40, 32, T(u8, 160), T(f16, 16), None, T(f32, 40), T(f32, 8), stream=0))
assert "scales" in refused(ValueError, lambda: dmv.pesti_gemv_i4group(8, 40, 32, T(u8, 160), T(f16, 15), None, T(f32, 40), T(f32, 8), stream=0))
cache = dmv.kv_cache("f16", 2, 8, 16, 2, 64, T(f16, 32768), T(f16, 32768))
table = dmv.kv_table(T(i32, 12), T(i32, 4), None, 4, 3)
refused(dmv.PestiError, lambda: dmv.pesti_cache_append(cache, table, 2, 3, Rows(f16, 3, 128), Rows(f16, 3, 128), stream=0))
assert "v must" in refused(ValueError, lambda: dmv.pesti_cache_append(cache, table, 2, 3, Rows(f16, 3, 128), Rows(f32, 3, 128), stream=0))
refused(dmv.PestiError, lambda: dmv.pesti_quant_i8token("f32", 2, 48, T(f32, 96), T(i8, 96), T(f32, 2), stream=0))
print("as documented")
"""


@pytest.mark.parametrize("other", ["", "1.0.0", "unsaid"])
def test_the_binding_without_the_argument_checks(other):
    source = WITHOUT.format(root=str(ROOT), tests=str(Path(__file__).resolve().parent), other=other)
    r = subprocess.run([sys.executable, "-c", source], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("as documented"), r.stdout + r.stderr


def test_the_compiled_checks_are_those_of_this_torch():
    """Where they were built they are bound, under this Python's own file name."""
    import torch
    from dequantize_mat_vec_amd import _lib
    _lib.load()
    fast = _lib._compiled()
    if fast is None:
        pytest.skip("not built here")
    assert fast.torch == torch.__version__ and _lib._sized is fast.sized
    assert Path(fast.__file__).name == build.ARGS_PATH.name
