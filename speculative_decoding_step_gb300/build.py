"""Build the CUDA library ``libpe.so`` (sm_103a) in-tree with nvcc.

Each translation unit is compiled in parallel, then linked into one shared
library exposing the C ABI declared in ``include/pe.h``.  ``pe_bind.so``, the Python
entry of the calls whose arguments would otherwise take longer than their work, is
compiled beside it against torch's headers (without torch the library is built alone).
"""

from __future__ import annotations

import concurrent.futures
import contextlib
import importlib.util
import os
import shutil
import subprocess
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(BUILD, "libpe.so")
BIND = os.path.join(BUILD, "pe_bind.so")
BIND_FOR = os.path.join(BUILD, "pe_bind.for")  # the torch and the Python that it was compiled against
SOURCES = ["pe_api.cu", "pe_meta.cu", "pe_gemm.cu", "pe_attn.cu", "pe_noalloc.cu", "pe_sample.cu", "pe_packed.cu",
           "pe_packed_attn.cu", "pe_mx.cu", "pe_mx_gemm.cu", "pe_mx_pair.cu", "pe_append.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", shutil.which("nvcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _flags():
    return ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", os.path.join(ROOT, "include"),
                   "-Xptxas", "-warn-spills"]


def _torch():
    """Where torch is installed; None where it is not."""
    spec = importlib.util.find_spec("torch")
    return spec.submodule_search_locations[0] if spec is not None else None


def _bind_command(torch: str, out: str):
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    include = [os.path.join(ROOT, "include"), sysconfig.get_paths()["include"], os.path.join(torch, "include"),
               os.path.join(cuda, "include")]
    return (["g++", "-O2", "-std=c++17", "-fPIC", "-shared"] + [f"-I{d}" for d in include] +
            [os.path.join(CSRC, "pe_bind.cpp"), "-o", out, "-L" + os.path.join(torch, "lib"), "-ltorch_python",
             "-ltorch_cpu", "-lc10", "-lc10_cuda"])


def _bind_for(torch: str) -> str:
    """What pe_bind.so is good for: it reads tensors' fields at the places that these headers give them."""
    with open(os.path.join(torch, "version.py")) as f:
        return "\n".join([torch, sysconfig.get_config_var("SOABI") or "", f.read()])


def bind_is_current() -> bool:
    """Whether pe_bind.so is there and was compiled against this torch and this Python."""
    torch = _torch()
    if torch is None or not os.path.exists(BIND) or not os.path.exists(BIND_FOR):
        return False
    with open(BIND_FOR) as f:
        return f.read() == _bind_for(torch)


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    headers = [os.path.join(CSRC, h) for h in os.listdir(CSRC) if h.endswith((".h", ".cuh"))]
    headers.append(os.path.join(ROOT, "include", "pe.h"))
    objs = []
    jobs = []
    for src in SOURCES:
        s = os.path.join(CSRC, src)
        o = os.path.join(BUILD, src.replace(".cu", ".o"))
        objs.append(o)
        if force or _stale(o, [s] + headers):
            jobs.append([nvcc()] + _flags() + ["-c", s, "-o", o])

    def run(cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"compiling failed: {' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
        return r.stderr

    bind_tmp, torch = BIND + f".tmp{os.getpid()}", _torch()
    # (a C caller needs libpe.so alone, and no torch)
    bind = torch is not None and (force or not bind_is_current() or
                                  _stale(BIND, [os.path.join(CSRC, "pe_bind.cpp"), os.path.join(ROOT, "include", "pe.h")]))
    if bind:
        jobs.append(_bind_command(torch, bind_tmp))
    with concurrent.futures.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        for log in ex.map(run, jobs):
            if verbose and log:
                print(log)
    if bind:
        # (a build that ends between these two compiles it again)
        with contextlib.suppress(FileNotFoundError):
            os.remove(BIND_FOR)
        os.replace(bind_tmp, BIND)
        with open(bind_tmp, "w") as f:
            f.write(_bind_for(torch))
        os.replace(bind_tmp, BIND_FOR)
    if _stale(LIB, objs):
        tmp = LIB + f".tmp{os.getpid()}"
        run([nvcc()] + ARCH + ["-shared", "-o", tmp] + objs)
        os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose=True))
