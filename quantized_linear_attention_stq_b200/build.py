"""Build the CUDA library in-tree: csrc/*.cu -> libstq.so (sm_100a only), and the binding's usual case:
csrc/binding.cpp -> _binding.so (host code against the installed torch).

``python -m quantized_linear_attention_stq_b200.build`` or ``build()`` from Python. The library
is rebuilt when a source or the public header is newer than the shared object.
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
HEADER = os.path.join(ROOT, "include", "stq.h")
LIB = os.path.join(PKG, "libstq.so")
BINDING = os.path.join(PKG, "_binding.so")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
         "--expt-relaxed-constexpr", "-Xptxas", "-warn-spills"]


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libstq.so")


def sources() -> list:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def stale() -> bool:
    if not os.path.exists(LIB):
        return True
    deps = sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + [HEADER]
    return os.path.getmtime(LIB) < max(os.path.getmtime(f) for f in deps)


def binding_key() -> str:
    """What the compiled module is built against: it reads torch's tensors through inlined code, so one
    built for another torch or Python must not be loaded, even where its symbols resolve."""
    import torch

    return f"torch {torch.__version__}, {sysconfig.get_config_var('SOABI')}"


def binding_stale() -> bool:
    src = os.path.join(CSRC, "binding.cpp")
    if not os.path.exists(BINDING) or os.path.getmtime(BINDING) < max(map(os.path.getmtime, (src, HEADER))):
        return True
    with open(BINDING, "rb") as f:  # the module holds its key as a string
        return binding_key().encode() + b"\0" not in f.read()


def build_binding(force: bool = False, verbose: bool = False) -> str:
    """Compile _binding.so where its source or the public header is newer, or it was built against another torch
    or Python. Returns "" (and warns) where there is no torch, host compiler or Python header to build with: the
    calls then go through ctypes."""
    try:
        import torch
    except ImportError:
        torch = None
    if torch is not None and not force and not binding_stale():
        return BINDING
    cxx, python_h = shutil.which("g++"), os.path.join(sysconfig.get_paths()["include"], "Python.h")
    missing = "torch" if torch is None else "g++" if cxx is None else "" if os.path.exists(python_h) else python_h
    if missing:
        warnings.warn(f"_binding.so is not built: {missing} is missing")
        return ""
    src, key = os.path.join(CSRC, "binding.cpp"), binding_key()
    root = os.path.dirname(torch.__file__)
    cuda = os.path.join(os.path.dirname(os.path.dirname(_nvcc())), "include")
    includes = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"), cuda,
                os.path.dirname(python_h)]
    tmp = BINDING + f".tmp{os.getpid()}"
    cmd = [cxx, "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", f'-DSTQ_BUILT_FOR="{key}"',
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *[f"-isystem{i}" for i in includes], "-o",
           tmp, src, "-L" + os.path.join(root, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python", "-L" + PKG,
           "-l:libstq.so", "-Wl,-rpath,$ORIGIN"]
    if verbose:
        print(" ".join(cmd), flush=True)
    proc = subprocess.run(cmd, capture_output=True, text=True)
    if proc.returncode != 0:
        raise RuntimeError(f"g++ failed on {src} ({proc.returncode}):\n{proc.stdout}\n{proc.stderr}")
    os.replace(tmp, BINDING)
    return BINDING


def _compile(src: str, obj: str, ptxas_info: bool):
    cmd = [_nvcc(), *ARCH, *FLAGS, "-c", "-o", obj, src]
    if ptxas_info:
        cmd += ["-Xptxas", "-v"]
    proc = subprocess.run(cmd, capture_output=True, text=True)
    return cmd, proc


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    """Compile every source to an object (in parallel, under the package's _build folder), then
    link libstq.so. Objects whose source and headers are older than them are reused."""
    if not (force or stale()):
        build_binding(force, verbose)
        return LIB
    from concurrent.futures import ThreadPoolExecutor

    objdir = os.path.join(ROOT, "_build", "stq")
    os.makedirs(objdir, exist_ok=True)
    headers = glob.glob(os.path.join(CSRC, "*.cuh")) + [HEADER]
    newest_header = max(os.path.getmtime(f) for f in headers)
    jobs = []
    for src in sources():
        obj = os.path.join(objdir, os.path.basename(src) + ".o")
        fresh = os.path.exists(obj) and os.path.getmtime(obj) >= max(os.path.getmtime(src), newest_header)
        jobs.append((src, obj, force or not fresh))
    todo = [j for j in jobs if j[2]]
    with ThreadPoolExecutor(max_workers=max(1, min(len(todo), os.cpu_count() or 1))) as ex:
        results = list(ex.map(lambda j: _compile(j[0], j[1], ptxas_info), todo))
    for (src, _, _), (cmd, proc) in zip(todo, results):
        if verbose:
            print(" ".join(cmd), flush=True)
        if proc.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src} ({proc.returncode}):\n{proc.stdout}\n{proc.stderr}")
        if verbose or ptxas_info:
            sys.stdout.write(proc.stdout + proc.stderr)
    tmp = LIB + f".tmp{os.getpid()}"
    link = [_nvcc(), *ARCH, "-shared", "-o", tmp, *[j[1] for j in jobs]]
    proc = subprocess.run(link, capture_output=True, text=True)
    if proc.returncode != 0:
        raise RuntimeError(f"nvcc link failed ({proc.returncode}):\n{proc.stdout}\n{proc.stderr}")
    os.replace(tmp, LIB)
    build_binding(force, verbose)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True, ptxas_info="--ptxas-info" in sys.argv)
