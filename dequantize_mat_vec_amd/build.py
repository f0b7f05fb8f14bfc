"""Build step: compile the HIP sources under csrc/ into libpesti.so (gfx950), and,
where a host compiler and torch's and Python's headers are there, the binding's
argument checks (without them the binding's own, in Python, do alone).

Run as `python -m dequantize_mat_vec_amd.build`; the package entry script's
build() calls the same function.  hipcc cross-compiles for gfx950 without a
GPU present.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig
from pathlib import Path

PKG_DIR = Path(__file__).resolve().parent
REPO = PKG_DIR.parent
SRC_DIR = PKG_DIR / "csrc"
INCLUDE_DIR = REPO / "include"
LIB_PATH = PKG_DIR / "libpesti.so"
# the binding's argument checks (host code), for this Python alone
ARGS_PATH = PKG_DIR / ("_tensor_args" + (sysconfig.get_config_var("EXT_SUFFIX") or ".so"))
ARCH = "gfx950"

# Packed float32 VALU ops are turned off for every device compilation; the
# host pass warns that it does not know the feature, which is harmless.
HIP_FLAGS = [
    f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC", "-shared",
    "-Wall", "-Wno-unused-command-line-argument",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
]


def hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), shutil.which("hipcc"), "/opt/rocm/bin/hipcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found: the HIP library cannot be built")


def sources():
    return sorted(SRC_DIR.glob("*.hip"))


def args_command(out: Path):
    """The host compiler's command for the binding's argument checks, against the installed torch."""
    import torch
    from torch.utils.cpp_extension import include_paths
    lib = Path(torch.__file__).resolve().parent / "lib"
    return [os.environ.get("CXX") or shutil.which("g++") or "c++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-D__HIP_PLATFORM_AMD__",
            f'-DPESTI_TORCH="{torch.__version__}"',
            f"-I{INCLUDE_DIR}", *[f"-isystem{p}" for p in (*include_paths(), "/opt/rocm/include", sysconfig.get_paths()["include"])],
            str(SRC_DIR / "tensor_args.cpp"), "-o", str(out), f"-L{lib}", "-ltorch_python", "-ltorch_cpu", "-lc10_hip", "-lc10"]


def start_args(out: Path):
    """The compilation of the argument checks, started, or why it could not be."""
    try:
        return subprocess.Popen(args_command(out), stdout=subprocess.PIPE, stderr=subprocess.STDOUT)
    except (ImportError, AttributeError, OSError) as e:   # no torch, one without these headers, no compiler
        return f"{type(e).__name__}: {e}"


def finish_args(started, out: Path) -> bool:
    """Put the argument checks in their place, or say why there are none; what an earlier build left goes either way."""
    text = started if isinstance(started, str) else started.communicate()[0].decode(errors="replace")
    for old in PKG_DIR.glob("_tensor_args*.so"):
        old.unlink()
    if isinstance(started, str) or started.returncode != 0:
        sys.stderr.write(f"--- tensor_args.cpp (left out: the binding checks its arguments in Python)\n{text}\n")
        out.unlink(missing_ok=True)
        return False
    os.replace(out, ARGS_PATH)
    return True


def build(verbose: bool = False) -> Path:
    """Compile every source into libpesti.so, and the binding's argument checks where that can be done (always recompiles)."""
    objs = []
    obj_dir = PKG_DIR / "_build"
    obj_dir.mkdir(exist_ok=True)
    procs = []
    args_tmp = obj_dir / "tensor_args.so.tmp"
    args = start_args(args_tmp)
    for src in sources():
        obj = obj_dir / (src.stem + ".o")
        cmd = [hipcc(), *[f for f in HIP_FLAGS if f != "-shared"], "-c", "-I", str(INCLUDE_DIR),
               str(src), "-o", str(obj)]
        if verbose:
            print(" ".join(cmd), flush=True)
        procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
        objs.append(obj)
    failed = []
    for src, p in procs:
        out, _ = p.communicate()
        text = out.decode(errors="replace")
        msgs = [ln for ln in text.splitlines() if "packed-fp32-ops" not in ln
                and "is not a recognized feature" not in ln]
        if p.returncode != 0:
            failed.append((src, text))
        elif verbose and any(m.strip() for m in msgs):
            print("\n".join(msgs), flush=True)
    if failed:
        for src, text in failed:
            sys.stderr.write(f"--- {src.name}\n{text}\n")
        if not isinstance(args, str):
            args.communicate()
        raise RuntimeError("HIP compilation failed")
    tmp = LIB_PATH.with_suffix(".so.tmp")
    cmd = [hipcc(), f"--offload-arch={ARCH}", "-shared", "-fPIC", "-o", str(tmp), *map(str, objs)]
    subprocess.run(cmd, check=True)
    finish_args(args, args_tmp)
    os.replace(tmp, LIB_PATH)
    return LIB_PATH


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
