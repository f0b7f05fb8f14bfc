"""The library's own rule for the kernel of an 8-bit or expert product
(csrc/tile_choice.h, plain C++), compiled for the host."""
from __future__ import annotations

import ctypes
import functools
import subprocess
import tempfile
from pathlib import Path

CSRC = Path(__file__).resolve().parent.parent / "dequantize_mat_vec_amd" / "csrc"
NAMES = ["rows 16", "rows 32", "rows 64", "64x128", "128x128", "128x256", "256x256"]
SOURCE = """
#include "tile_choice.h"
using namespace pesti_host;
extern "C" int kernel_of(long long rows, long long n, long long experts, long long kbytes, int gated) {
  return static_cast<int>(tile_kernel(TileShape{rows, n, experts, kbytes, gated != 0}));
}
extern "C" int wavefronts_of(long long kbytes) { return rows_wavefronts(kbytes); }
extern "C" long long workgroups_of(long long experts, long long bm, long long bn) {
  return tile_workgroups(TileShape{0, 0, experts, 0, false}, bm, bn);
}
"""


@functools.lru_cache(maxsize=None)
def library():
    with tempfile.TemporaryDirectory() as d:
        src, so = Path(d) / "tile_choice.cpp", Path(d) / "tile_choice_host.so"
        src.write_text(SOURCE)
        subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I", str(CSRC), str(src), "-o", str(so)], check=True)
        lib = ctypes.CDLL(str(so))   # stays mapped after the folder is gone
    ll = ctypes.c_longlong
    lib.kernel_of.argtypes = [ll, ll, ll, ll, ctypes.c_int]
    lib.workgroups_of.argtypes = [ll, ll, ll]
    lib.workgroups_of.restype = ll
    lib.wavefronts_of.argtypes = [ll]
    return lib


def kernel(rows, n, k, form, experts=0, gated=False):
    """Name of the kernel; experts = 0 for the dense call."""
    return NAMES[library().kernel_of(rows, n, experts, k * (2 if form == "f16" else 1), int(gated))]


def wavefronts(k, form):
    return library().wavefronts_of(k * (2 if form == "f16" else 1))


def tiles_and_workgroups(name, counts, n, experts, gated=False):
    """Tiles that the rows of these counts come to, and the workgroups that take them in turn."""
    bm, bn = (int(v) for v in name.split("x"))
    cols = bn // 2 if gated else bn
    return sum(-(-c // bm) for c in counts) * -(-n // cols), library().workgroups_of(experts, bm, bn)
