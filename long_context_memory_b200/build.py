"""Build libmsa.so (the C-ABI library) in-tree with nvcc for sm_100a, and _fastcall (the binding's checks
of latency-bound calls) with the host compiler against PyTorch's headers.  The library needs nvcc alone:
without PyTorch it is built, and the binding's part is left out."""
from __future__ import annotations

import importlib.util
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
SOURCES = ["msa_api.cu", "route.cu", "route_static.cu", "attend.cu", "encode.cu", "aux_loss.cu", "tiered.cu",
           "rotary.cu", "tree.cu"]
LIB = os.path.join(HERE, "libmsa.so")
FAST = os.path.join(HERE, "_fastcall.so")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")


def needs_build() -> bool:
    built = [LIB] + ([FAST] if importlib.util.find_spec("torch") else [])
    if not all(os.path.exists(f) for f in built):
        return True
    t = min(os.path.getmtime(f) for f in built)
    deps = [os.path.join(CSRC, f) for f in os.listdir(CSRC)] + [os.path.join(ROOT, "include", "msa.h")]
    return any(os.path.getmtime(p) > t for p in deps)


def fastcall_command() -> list:
    """The compiler command of _fastcall.so."""
    import sysconfig

    import torch
    from torch.utils import cpp_extension

    cuda = os.path.dirname(os.path.dirname(NVCC))
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    return ([os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-w",
             f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"]
            + [f"-I{d}" for d in cpp_extension.include_paths() + [os.path.join(cuda, "include"),
                                                                  sysconfig.get_paths()["include"]]]
            + [os.path.join(CSRC, "fastcall.cpp"), "-o", FAST, f"-L{lib}", "-ltorch_python", "-ltorch_cpu", "-lc10",
               "-lc10_cuda", "-ldl"])


def build(verbose: bool = False, ptxas_verbose: bool = False) -> str:
    """Compile every source to an object in parallel (relocatable device code), then link libmsa.so;
    beside them _fastcall.so, whose failure is raised once the library stands."""
    import concurrent.futures as cf
    import tempfile

    flags = [NVCC, "-O3", "-std=c++17", "-gencode", "arch=compute_100a,code=sm_100a", "-lineinfo", "-rdc=true",
             "-Xcompiler", "-fPIC", "-I", os.path.join(ROOT, "include")]
    if ptxas_verbose:
        flags += ["-Xptxas", "-v"]
    with tempfile.TemporaryDirectory(prefix="msa_build_") as tmp:
        objs = [os.path.join(tmp, os.path.splitext(src)[0] + ".o") for src in SOURCES]
        cmds = [flags + ["-c", os.path.join(CSRC, src), "-o", obj] for src, obj in zip(SOURCES, objs)]
        try:
            cmds.append(fastcall_command())
        except ImportError as e:
            sys.stderr.write(f"_fastcall.so is left out ({e}): the binding's rotation, norm and draft-tree calls need it\n")
        if verbose:
            for c in cmds:
                print(" ".join(c), flush=True)
        with cf.ThreadPoolExecutor(max_workers=len(cmds)) as ex:
            results = list(ex.map(lambda c: subprocess.run(c, capture_output=True, text=True), cmds))
        for r in results:
            if r.returncode != 0:
                sys.stderr.write(r.stdout + r.stderr)
            elif verbose or ptxas_verbose:
                sys.stderr.write(r.stderr)
        if any(r.returncode != 0 for r in results[:len(objs)]):
            raise RuntimeError("nvcc failed building libmsa.so")
        link = [NVCC, "-gencode", "arch=compute_100a,code=sm_100a", "-rdc=true", "-shared", "-Xcompiler", "-fPIC",
                "-cudart", "static", "-o", LIB] + objs
        if verbose:
            print(" ".join(link), flush=True)
        r = subprocess.run(link, capture_output=True, text=True)
        if r.returncode != 0:
            sys.stderr.write(r.stdout + r.stderr)
            raise RuntimeError("nvcc failed linking libmsa.so")
        if any(r.returncode != 0 for r in results[len(objs):]):
            raise RuntimeError("libmsa.so is built, but compiling _fastcall.so failed")
    return LIB


if __name__ == "__main__":
    build(verbose=True, ptxas_verbose="-v" in sys.argv)
    print(LIB)
