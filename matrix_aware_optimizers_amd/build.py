"""Build libmao.so (the HIP/gfx950 library) in place next to this file.

Usage: ``python -m matrix_aware_optimizers_amd.build`` (or call ``build()``).
Every ``.hip`` file under ``csrc/`` is compiled to an object with hipcc for
gfx950 and the objects are linked into ``libmao.so``. Objects go to
``_build/`` at the repository root. ``csrc/binding.cpp`` (host code: torch
tensors to the C ABI, for the layer operators) becomes ``_layers.so`` beside it,
where g++, torch's headers and Python's are there; the library needs hipcc alone.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
OBJ = os.path.join(ROOT, "_build")
LIB = os.path.join(HERE, "libmao.so")
BINDING = os.path.join(HERE, "_layers.so")

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
ARCH = "gfx950"
FLAGS = [
    f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC", "-fvisibility=hidden",
    # packed-fp32 instructions stay off on this target
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wno-unused-command-line-argument",
]


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".hip"))


def _compile(src: str) -> str:
    obj = os.path.join(OBJ, os.path.basename(src) + ".o")
    cmd = [HIPCC, *FLAGS, "-I", os.path.join(ROOT, "include"), "-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed on {src}:\n{r.stdout}\n{r.stderr}")
    return obj


def _run(cmd, what):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stdout}\n{r.stderr}")


def _binding_lacks():
    """What csrc/binding.cpp needs and this machine does not have, or None."""
    if shutil.which("g++") is None:
        return "g++"
    try:
        import torch
    except ImportError:
        return "torch"
    inc = os.path.join(os.path.dirname(torch.__file__), "include", "ATen", "core", "Tensor.h")
    if not os.path.exists(inc):
        return "torch's headers"
    if not os.path.exists(os.path.join(sysconfig.get_paths()["include"], "Python.h")):
        return "Python's headers"
    return None


def _compile_binding() -> str:
    """The object of csrc/binding.cpp."""
    import torch
    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    obj = os.path.join(OBJ, "binding.o")
    _run(["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-c",
          f"-I{inc}", f"-I{inc}/torch/csrc/api/include", f"-I{sysconfig.get_paths()['include']}",
          f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
          os.path.join(CSRC, "binding.cpp"), "-o", obj], "g++ on binding.cpp")
    return obj


def _link_binding(obj: str):
    import torch
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = BINDING + ".tmp"
    _run(["g++", "-shared", "-o", tmp, obj, LIB, f"-L{lib}", "-ltorch_python", "-ltorch_cpu",
          "-lc10", "-Wl,-rpath,$ORIGIN"], "link of _layers.so")
    shutil.move(tmp, BINDING)


def build(verbose: bool = False) -> str:
    """Compile every HIP source for gfx950 and link libmao.so; returns its path. Then
    the binding of the layer calls, _layers.so: left out, and said so, where its
    compiler or headers are missing; an error in it is raised with the library built."""
    if not os.path.exists(HIPCC):
        raise RuntimeError(f"hipcc not found at {HIPCC}")
    os.makedirs(OBJ, exist_ok=True)
    srcs = sources()
    workers = min(len(srcs), max(1, (os.cpu_count() or 2) // 2))
    lacks = _binding_lacks()
    with cf.ThreadPoolExecutor(max_workers=workers) as ex:
        binding = None if lacks else ex.submit(_compile_binding)
        objs = list(ex.map(_compile, srcs))
    tmp = LIB + ".tmp"
    _run([HIPCC, f"--offload-arch={ARCH}", "-shared", "-fPIC", "-Wl,-soname,libmao.so", "-o", tmp,
          *objs], "link of libmao.so")
    shutil.move(tmp, LIB)
    if os.path.exists(BINDING):  # of the library before
        os.remove(BINDING)
    if lacks:
        print(f"built {LIB} without _layers.so (the Python layer calls): no {lacks}",
              file=sys.stderr)
        return LIB
    _link_binding(binding.result())
    if verbose:
        print(f"built {LIB}")
    return LIB


if __name__ == "__main__":
    build(verbose=True)
    sys.exit(0)
