"""Builds libdsv.so in-tree for sm_103a (nvcc, no cmake), and the native
binding of the row calls (_rows.so, the host compiler against torch's headers).

Each CUDA translation unit is compiled in parallel into ``_build/`` and linked
into ``dynamic_sparse_attention_dsv_gb300/libdsv.so`` against the shared CUDA
runtime; the binding links against it. ``python -m dynamic_sparse_attention_dsv_gb300.build`` runs it.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libdsv.so")
BINDING = os.path.join(PKG, "_rows.so")
SOURCES = ["host_common.cu", "lowrank_topk.cu", "attn_fwd.cu", "attn_bwd.cu", "rows_host.cu", "row_norm_fwd.cu",
           "row_norm_bwd.cu", "act_pack.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ARCH + ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
                "-I" + os.path.join(ROOT, "include")]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _cuda_lib_dir(nvcc: str) -> str:
    root = os.path.dirname(os.path.dirname(os.path.realpath(nvcc)))
    for sub in ("lib64", "lib", os.path.join("targets", "sbsa-linux", "lib"),
                os.path.join("targets", "x86_64-linux", "lib")):
        d = os.path.join(root, sub)
        if os.path.exists(os.path.join(d, "libcudart.so")):
            return d
    return os.path.join(root, "lib64")


def _stale(out: str, deps) -> bool:
    if not os.path.exists(out):
        return True
    t = os.path.getmtime(out)
    return any(os.path.getmtime(d) > t for d in deps)


def _binding_cmds(nvcc: str):
    """Compiling and linking the native binding."""
    import torch
    from torch.utils import cpp_extension

    torch_lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "include")
    obj = os.path.join(BUILD, "rows_binding.o")
    inc = cpp_extension.include_paths() + [sysconfig.get_paths()["include"], cuda]
    compile_ = ["g++", "-O2", "-std=c++17", "-fPIC", "-Wall",
                f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"]
    for d in inc:
        compile_ += ["-isystem", d]
    compile_ += ["-c", os.path.join(CSRC, "rows_binding.cpp"), "-o", obj]
    link = ["g++", "-shared", "-o", BINDING, obj, "-L" + PKG, "-l:libdsv.so", "-L" + torch_lib, "-lc10",
            "-lc10_cuda", "-ltorch_cpu", "-ltorch", "-ltorch_python", "-Wl,-rpath,$ORIGIN", "-Wl,-rpath," + torch_lib]
    return compile_, link, obj


def build(force: bool = False, verbose: bool = False) -> str:
    """Compiles and links libdsv.so and the binding; returns libdsv.so's path. Raises on failure."""
    nvcc = _nvcc()
    os.makedirs(BUILD, exist_ok=True)
    headers = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    headers.append(os.path.join(ROOT, "include", "libdsv.h"))
    objs = []
    jobs = []
    for src in SOURCES:
        s = os.path.join(CSRC, src)
        o = os.path.join(BUILD, src.replace(".cu", ".o"))
        objs.append(o)
        if force or _stale(o, [s] + headers):
            jobs.append([nvcc] + FLAGS + ["-c", s, "-o", o])

    def run(cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("compiling failed:\n" + " ".join(cmd) + "\n" + r.stdout + r.stderr)
        if verbose:
            sys.stdout.write(r.stdout + r.stderr)

    bind, bind_link, bind_obj = _binding_cmds(nvcc)
    bind_stale = force or _stale(bind_obj, [os.path.join(CSRC, "rows_binding.cpp"),
                                            os.path.join(ROOT, "include", "libdsv.h")])
    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        list(ex.map(run, jobs + ([bind] if bind_stale else [])))
    if force or jobs or _stale(LIB, objs):
        libdir = _cuda_lib_dir(nvcc)
        run([nvcc] + ARCH + ["-shared", "-cudart", "shared", "-o", LIB] + objs +
            ["-L" + libdir, "-Xlinker", "-rpath=" + libdir])
    if bind_stale or _stale(BINDING, [bind_obj, LIB]):
        run(bind_link)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
