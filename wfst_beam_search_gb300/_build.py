"""Compile the CUDA decoder library for GB300 (sm_103a), in tree.

Ten translation units are compiled in parallel and linked into
``wfst_beam_search_gb300/_build/libwfst_gb300.so``.  Where torch with CUDA and
Python's headers are installed, ``ops_binding.so`` is compiled beside it: the
second-pass operators' path from torch tensors into that library.
"""
from __future__ import annotations

import importlib.util
import os
import shutil
import subprocess
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(BUILD, "libwfst_gb300.so")
BINDING = os.path.join(BUILD, "ops_binding.so")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
SOURCES = ["wfst_kernel.cu", "wfst_api.cu", "wfst_static.cu", "wfst_preslice.cu", "wfst_vmm.cu", "wfst_probe.cu",
           "wfst_matvec.cu", "wfst_rotate.cu", "wfst_attend.cu", "wfst_sample.cu"]
BINDING_SOURCE = "ops_binding.cpp"
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA decoder cannot be built")


def _torch():
    """torch's folder; None where it, its CUDA part or Python's headers are missing, and the decoder is built alone."""
    spec = importlib.util.find_spec("torch")
    if not (spec and spec.origin and os.path.exists(os.path.join(sysconfig.get_paths()["include"], "Python.h"))):
        return None
    folder = os.path.dirname(spec.origin)
    needed = ("lib/libc10_cuda.so", "lib/libtorch_cuda.so", "include/c10/cuda/CUDAStream.h")
    return folder if all(os.path.exists(os.path.join(folder, *n.split("/"))) for n in needed) else None


def _made_for(torch):
    """What the binding's binary interface goes by: this Python and this torch."""
    with open(os.path.join(torch, "version.py")) as f:
        return f"{sysconfig.get_config_var('SOABI')}\n{torch}\n{f.read()}"


def _stamp():
    try:
        with open(BINDING + ".made_for") as f:
            return f.read()
    except OSError:
        return None


def _inputs():
    files = [os.path.join(CSRC, s) for s in SOURCES + [BINDING_SOURCE]]
    files += [os.path.join(CSRC, "wfst_internal.h"), os.path.join(CSRC, "wfst_vmm.h"),
              os.path.join(CSRC, "wfst_ops.h"),
              os.path.join(INCLUDE, "wfst_gb300.h")]
    return files


def up_to_date() -> bool:
    torch = _torch()
    made = [LIB, BINDING] if torch else [LIB]
    if not all(map(os.path.exists, made)) or (torch and _stamp() != _made_for(torch)):
        return False
    t = min(map(os.path.getmtime, made))
    return all(os.path.getmtime(f) <= t for f in _inputs())


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and up_to_date():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()
    flags = ARCH + ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-I", INCLUDE]
    if verbose:
        flags += ["-Xptxas", "-v"]

    torch = _torch()
    binding_flags = ["-O2", "-std=c++17", "-Xcompiler", "-fPIC", "-I", sysconfig.get_paths()["include"]]
    if torch:
        binding_flags += ["-I", os.path.join(torch, "include"),
                          "-I", os.path.join(torch, "include", "torch", "csrc", "api", "include")]

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
        cmd = [cc] + (binding_flags if src == BINDING_SOURCE else flags) + ["-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        return obj, r.stderr

    sources = SOURCES + ([BINDING_SOURCE] if torch else [])
    with ThreadPoolExecutor(max_workers=len(sources)) as ex:
        results = list(ex.map(compile_one, sources))
    objs = [o for o, _ in results[:len(SOURCES)]]
    tmp = LIB + f".{os.getpid()}.tmp"
    cmd = [cc] + ARCH + ["-shared", "-o", tmp] + objs + ["-lcudart"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    if torch:
        tmp = BINDING + f".{os.getpid()}.tmp"
        cmd = [cc] + ARCH + ["-shared", "-o", tmp, results[-1][0], "-L", BUILD, "-lwfst_gb300",
                             "-L", os.path.join(torch, "lib"), "-ltorch_python", "-ltorch_cuda", "-ltorch_cpu", "-ltorch",
                             "-lc10_cuda", "-lc10", "-Xlinker", "-rpath,$ORIGIN"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, BINDING)
        with open(BINDING + ".made_for", "w") as f:
            f.write(_made_for(torch))
    if verbose:
        for _, log in results:
            print(log)
    return LIB
