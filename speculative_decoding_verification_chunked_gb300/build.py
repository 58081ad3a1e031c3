"""Builds the CUDA library ``libsvx.so`` in-tree for sm_103a, and its bounds-checked
variant ``libsvx_checked.so`` (-DSVX_BOUNDS_CHECK: every kernel checks its global
accesses against the buffers its launch describes and reports a stray one through
the device error word instead of making it).

Each translation unit is compiled by its own nvcc process (all in parallel), then
linked into one shared library next to this file.  The binding's native part,
``svx_torch.so`` (a Python extension against this machine's PyTorch), is compiled beside them;
the libraries need no PyTorch and are built without it too.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libsvx.so")
LIB_CHECKED = os.path.join(PKG, "libsvx_checked.so")
LIB_TORCH = os.path.join(PKG, "svx_torch.so")

SOURCES = ["svx_kernels.cu", "svx_tc_kernel.cu", "svx_runtime.cu", "svx_static.cu", "svx_tier.cu", "svx_sched.cu", "svx_width.cu",
           "svx_paged.cu", "svx_heads.cu", "svx_decode.cu", "svx_evict.cu",
           "svx_residual.cu", "svx_cross.cu", "svx_shared.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
         "-Xcompiler", "-ffp-contract=off",
         "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libsvx.so")


def torch_command(out: str) -> list:
    """The compiler call that makes svx_torch.so."""
    import sysconfig

    import torch
    if torch.version.cuda is None:
        raise ImportError("this PyTorch is built without CUDA")
    home = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    includes = [os.path.join(home, "include"), os.path.join(home, "include", "torch", "csrc", "api", "include"),
                sysconfig.get_paths()["include"], os.path.join(cuda, "include"), INCLUDE]
    lib = os.path.join(home, "lib")
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            *[x for d in includes for x in ("-isystem" if d != INCLUDE else "-I", d)], os.path.join(CSRC, "svx_torch.cpp"), "-o", out,
            "-L", lib, f"-Wl,-rpath,{lib}", "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10"]


def build(verbose: bool = False, extra_flags: tuple = (), checked: bool = True) -> str:
    """Compiles every translation unit (both variants at once when `checked`) and links libsvx.so, then
    libsvx_checked.so; svx_torch.so too where PyTorch with CUDA is installed (else the binding's calls that need it raise
    ImportError).  A failure to compile svx_torch.so is raised once the libraries are linked.  Returns the path
    of libsvx.so."""
    cc = nvcc()
    variants = [("", LIB, ())] + ([("checked", LIB_CHECKED, ("-DSVX_BOUNDS_CHECK",))] if checked else [])
    procs, objs = [], {}
    for sub, lib, flags in variants:
        bdir = os.path.join(BUILD, sub) if sub else BUILD
        os.makedirs(bdir, exist_ok=True)
        for src in SOURCES:
            obj = os.path.join(bdir, src.replace(".cu", ".o"))
            cmd = [cc, *ARCH, *FLAGS, *flags, *extra_flags, "-c", os.path.join(CSRC, src), "-o", obj]
            if verbose:
                print(" ".join(cmd), file=sys.stderr)
            procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)))
            objs.setdefault(lib, []).append(obj)
    binding, why = None, ""
    try:
        cmd = torch_command(LIB_TORCH + ".tmp")
        if verbose:
            print(" ".join(cmd), file=sys.stderr)
        binding = subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    except ImportError as e:
        print(f"svx_torch.so is not built: {e}", file=sys.stderr)
    except OSError as e:  # no host compiler of that name
        why = str(e)
    failed = []

    def finish(src, p):
        out, _ = p.communicate()
        if p.returncode != 0:
            failed.append(f"--- {src}\n{out}")
        elif verbose and out.strip():
            print(out, file=sys.stderr)
    for src, p in procs:
        finish(src, p)
    if failed:
        if binding:
            binding.communicate()
        raise RuntimeError("compilation failed:\n" + "\n".join(failed))
    for _sub, lib, _flags in variants:
        tmp = lib + ".tmp"
        cmd = [cc, *ARCH, "-shared", "-o", tmp, *objs[lib]]
        r = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
        if r.returncode != 0:
            raise RuntimeError("link failed:\n" + r.stdout)
        os.replace(tmp, lib)
    if binding:
        finish("svx_torch.cpp", binding)
        if not failed:
            os.replace(LIB_TORCH + ".tmp", LIB_TORCH)
            return LIB
    # no binding of an earlier build beside new libraries
    if os.path.exists(LIB_TORCH):
        os.remove(LIB_TORCH)
    if failed or why:
        raise RuntimeError("the libraries are built; svx_torch.so is not:\n" + "\n".join(failed or [why]))
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
