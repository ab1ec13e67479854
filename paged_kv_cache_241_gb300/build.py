"""Build the pkv CUDA library in-tree (sm_103a only).

    python -m paged_kv_cache_241_gb300.build

Compiles every csrc/*.cu (and the host-only *.cpp) in parallel with nvcc and
links libpkv.so next to this file; beside it the C++ part of the Python binding
(csrc/pycall.cc), for the interpreter and the torch that run this (left out where torch is
missing or without CUDA).  No CMake; a rebuild only recompiles sources newer than their object.
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
INCLUDE = os.path.join(ROOT, "include")
OBJ_DIR = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libpkv.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found; the pkv library needs the CUDA toolkit")
    return cand


def _headers_mtime() -> float:
    hs = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    hs.append(os.path.join(INCLUDE, "pkv.h"))
    return max(os.path.getmtime(h) for h in hs)


def _compile(src: str, extra: list[str]) -> str:
    obj = os.path.join(OBJ_DIR, os.path.splitext(os.path.basename(src))[0] + ".o")
    if os.path.exists(obj) and os.path.getmtime(obj) >= max(os.path.getmtime(src), _headers_mtime()):
        return obj
    cmd = [nvcc(), *ARCH, *FLAGS, *extra, "-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    if r.stderr.strip():
        sys.stderr.write(r.stderr)
    return obj


def call_module() -> str:
    """Where the C++ part of the binding is for this interpreter."""
    return os.path.join(HERE, "_pkv_call" + (sysconfig.get_config_var("EXT_SUFFIX") or ".so"))


def _build_call_module() -> None:
    try:
        import torch
    except ImportError:
        torch = None
    if torch is None or torch.version.cuda is None:
        # (the rest of the library needs neither)
        sys.stderr.write("the binding's C++ part is left out: "
                         + ("no torch\n" if torch is None else "this torch has no CUDA\n"))
        return
    src, out = os.path.join(CSRC, "pycall.cc"), call_module()
    home = os.path.dirname(torch.__file__)
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        raise RuntimeError("no C++ compiler for the Python binding")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")
    cmd = [cxx, "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           f'-DPKV_TORCH_VERSION="{torch.__version__}"',
           "-I", sysconfig.get_paths()["include"], "-I", INCLUDE,
           "-isystem", os.path.join(home, "include"), "-isystem", cuda, src, "-o", out,
           "-L", os.path.join(home, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"]
    # Beside the objects, the command that made the module: with another torch, interpreter or
    # toolkit it is another one, whatever their files' times say.
    made_by = os.path.join(OBJ_DIR, os.path.basename(out) + ".txt")
    inputs = [src, os.path.join(INCLUDE, "pkv.h"), os.path.join(home, "version.py")]
    if os.path.exists(out) and os.path.exists(made_by):
        with open(made_by) as f:
            same = f.read() == repr(cmd)
        if same and os.path.getmtime(out) >= max(map(os.path.getmtime, inputs)):
            return
        os.remove(made_by)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{cxx} failed for {src}:\n{r.stdout}\n{r.stderr}")
    with open(made_by, "w") as f:
        f.write(repr(cmd))


def build(verbose_ptxas: bool = False) -> str:
    os.makedirs(OBJ_DIR, exist_ok=True)
    srcs = sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cu", ".cpp")))
    extra = ["-Xptxas", "-v"] if verbose_ptxas else []
    with cf.ThreadPoolExecutor(max_workers=8) as ex:
        call = ex.submit(_build_call_module)
        objs = list(ex.map(lambda s: _compile(s, extra), srcs))
    newest = max(os.path.getmtime(o) for o in objs)
    if not os.path.exists(LIB) or os.path.getmtime(LIB) < newest:
        cmd = [nvcc(), *ARCH, "-shared", "-o", LIB, *objs]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    call.result()  # (its error, with the library in place)
    return LIB


if __name__ == "__main__":
    print(build(verbose_ptxas="-v" in sys.argv))
