"""Build libmq.so (the C-ABI library of include/mq.h) in-tree for sm_103a.

nvcc compiles every translation unit of csrc/ in parallel (one -gencode,
sm_103a only, no fast-math so that the producers' IEEE division, reciprocal
and rounding match the definition), then links a shared library against the
shared CUDA runtime.  Output: quant_quantized_gemv_gb300/_build/libmq.so.
That needs nvcc alone.  Beside it, where torch is installed, a Python module over
its headers with the calls of the operators that name many tensors
(csrc/binding.cpp), in a file named after the Python and the torch it is for.
"""
from __future__ import annotations

import os
import re
import shutil
import subprocess
import sysconfig
from concurrent.futures import ThreadPoolExecutor
from importlib.util import find_spec

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
SO = os.path.join(BUILD, "libmq.so")
SOURCES = ["gemv.cu", "gemv_batch.cu", "gemv_gateup.cu", "gemv_f32.cu", "producers.cu", "noalloc.cu",
           "readfloor.cu", "copy.cu", "repack_device.cu", "rope_append.cu", "attn_decode.cu", "sample.cu",
           "api.cpp", "repack.cpp", "decode.cpp"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else (shutil.which("nvcc") or "nvcc")


def _torch() -> tuple[str, str] | None:
    """Where torch lies and its version, without an import; None where there is none."""
    spec = find_spec("torch")
    path = spec.submodule_search_locations[0] if spec and spec.submodule_search_locations else ""
    version = os.path.join(path, "version.py")
    if not path or not os.path.exists(version):  # none, or a folder of that name
        return None
    with open(version) as f:
        return path, re.search(r"^__version__\s*=\s*['\"]([^'\"]+)", f.read(), re.M)[1]


def binding() -> str | None:
    """The module of the Python calls for this Python and torch; None without torch."""
    torch = _torch()
    return torch and os.path.join(BUILD, f"mq_binding.{sysconfig.get_config_var('SOABI')}.torch-{torch[1]}.so")


def _stale() -> bool:
    made = [f for f in (SO, binding()) if f]
    if not all(os.path.exists(f) for f in made):
        return True
    t = min(os.path.getmtime(f) for f in made)
    deps = [os.path.join(CSRC, f) for f in os.listdir(CSRC)] + [os.path.join(INCLUDE, "mq.h")]
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and not _stale():
        return SO
    os.makedirs(BUILD, exist_ok=True)
    common = ["-O3", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC]

    def compile_one(src: str) -> str:
        obj = os.path.join(BUILD, src + ".o")
        cmd = [nvcc(), *common, "-c", os.path.join(CSRC, src), "-o", obj]
        if src.endswith(".cu"):
            cmd[1:1] = [*ARCH, "-lineinfo", "-Xptxas", "-v" if verbose else "-O3"]
        if src == "binding.cpp":
            headers = [os.path.join(torch, "include"), os.path.join(torch, "include", "torch", "csrc", "api", "include"),
                       sysconfig.get_paths()["include"],
                       os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")]
            cmd[1:1] = [x for h in headers for x in ("-I", h)]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr)
        return obj

    def link(so: str, objs: list, libs: list):
        tmp = so + f".{os.getpid()}.tmp"
        cmd = [nvcc(), *ARCH, "-shared", "-cudart", "shared", "-o", tmp, *objs, *libs]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, so)

    so, torch = binding(), (_torch() or [None])[0]
    with ThreadPoolExecutor(len(SOURCES) + 1) as ex:
        calls = ex.submit(compile_one, "binding.cpp") if so else None
        link(SO, list(ex.map(compile_one, SOURCES)), [])
    if calls:
        lib = os.path.join(torch, "lib")
        link(so, [calls.result()], ["-L", lib, "-Xlinker", "-rpath", "-Xlinker", lib, "-ltorch_python", "-ltorch_cpu",
                                    "-lc10_cuda", "-lc10"])
    return SO


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
