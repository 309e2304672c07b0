"""Build libmoe_decode.so in-tree for sm_103a (nvcc, one object per source,
compiled in parallel, then linked), and beside it, where torch is installed,
_calls.so, the extension module through which Python makes the attention
operators' calls.  The library itself needs nvcc alone.
Usage: python -m moe_decode_layer_bf16_gb300.build"""

from __future__ import annotations

import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libmoe_decode.so")
CALLS = os.path.join(PKG, "_calls.so")
SOURCES = ["api.cu", "gemv.cu", "experts.cu", "experts_tc.cu", "rmsnorm.cu", "mtp.cu",
           "api_attention.cu", "fp8_linear.cu", "kv_append.cu", "attention.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--threads", "1"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _read(path: str):
    if not os.path.exists(path):
        return None
    with open(path) as f:
        return f.read()


def _newer(target: str, deps) -> bool:
    if not os.path.exists(target):
        return False
    t = os.path.getmtime(target)
    return all(os.path.getmtime(d) <= t for d in deps)


def _torch_root():
    """Where torch is, without importing it; None if it is not installed."""
    import importlib.util
    spec = importlib.util.find_spec("torch")
    return os.path.dirname(spec.origin) if spec and spec.origin else None


def _calls_key() -> str:
    """What the extension module is compiled against, beside its sources."""
    root = _torch_root()
    return f"torch in {root}:\n{_read(os.path.join(root, 'version.py'))}\nPython {sys.version}\n"


def calls_command(source: str, obj: str):
    """Compiles calls.cpp against this interpreter's and this torch's headers."""
    import sysconfig
    inc = os.path.join(_torch_root(), "include")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")
    dirs = [inc, os.path.join(inc, "torch", "csrc", "api", "include"), sysconfig.get_paths()["include"], cuda]
    return [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", *("-I" + d for d in dirs), "-c", source, "-o", obj]


def build(verbose: bool = False, extra_flags=None) -> str:
    os.makedirs(BUILD, exist_ok=True)
    headers = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".h", ".cuh"))]
    headers.append(os.path.join(PKG, "..", "include", "moe_decode.h"))
    cc = nvcc()
    extra = list(extra_flags or [])
    key_file = os.path.join(BUILD, "calls.key")
    torch_root = _torch_root()

    def compile_one(src):
        s = os.path.join(CSRC, src)
        o = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
        python = src.endswith(".cpp")
        if _newer(o, [s, *headers]) and not extra and (not python or _read(key_file) == _calls_key()):
            return o
        cmd = calls_command(s, o) if python else [cc, *ARCH, *FLAGS, *extra, "-c", s, "-o", o]
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"{os.path.basename(cmd[0])} failed for {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout, r.stderr, flush=True)
        if python:
            with open(key_file, "w") as f:
                f.write(_calls_key())
        return o

    def link(target, objs, cmd):
        if _newer(target, objs):
            return
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")

    with ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        calls = ex.submit(compile_one, "calls.cpp") if torch_root else None
        objs = list(ex.map(compile_one, SOURCES))
        link(LIB, objs, [cc, *ARCH, "-shared", "-o", LIB, *objs])
    if calls:
        obj, libs = calls.result(), os.path.join(torch_root, "lib")
        link(CALLS, [obj, LIB],
             [os.environ.get("CXX", "g++"), "-shared", "-o", CALLS, obj, "-L" + libs, "-ltorch_python", "-ltorch",
              "-ltorch_cpu", "-lc10", "-lc10_cuda", "-L" + PKG, "-l:libmoe_decode.so", "-Wl,-rpath,$ORIGIN",
              "-Wl,-rpath," + libs])
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
