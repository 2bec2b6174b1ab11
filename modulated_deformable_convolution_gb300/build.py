"""Builds libmdcn.so in-tree with nvcc for sm_103a (no cmake), and beside it
_token_binding.so, the binding of the operators on tokens, with g++.

    python -m modulated_deformable_convolution_gb300.build [--force]

The library needs nvcc alone; a binding that does not build (no g++, no headers
of Python or torch) is an error after the library has been linked.

Objects go to ``_build/`` beside this file; translation units compile in
parallel; ptxas resource usage (registers, shared memory, spills) is written
to ``_build/ptxas.log``.
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libmdcn.so")
BINDING_SOURCE = os.path.join(CSRC, "mdcn_token_binding.cpp")
BINDING = os.path.join(HERE, "_token_binding.so")

CU_SOURCES = ["mdcn_fused.cu", "mdcn_prep.cu", "mdcn_im2col.cu", "mdcn_noalloc.cu", "mdcn_backward.cu", "mdcn_gemm.cu",
              "mdcn_direct.cu", "mdcn_rotary.cu", "mdcn_attention_simt.cu",
              "mdcn_attention_tc.cu", "mdcn_attention_tc_backward.cu"]
CPP_SOURCES = ["mdcn_api.cpp", "mdcn_attention_api.cpp"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def cuda_home() -> str:
    for cand in (os.environ.get("CUDA_HOME"), os.environ.get("CUDA_PATH"), "/usr/local/cuda"):
        if cand and os.path.exists(os.path.join(cand, "bin", "nvcc")):
            return cand
    nvcc = shutil.which("nvcc")
    if nvcc:
        return os.path.dirname(os.path.dirname(nvcc))
    raise RuntimeError("nvcc not found (set CUDA_HOME)")


def _headers():
    out = []
    for d in (CSRC, INCLUDE):
        for f in os.listdir(d):
            if f.endswith((".h", ".cuh")):
                out.append(os.path.join(d, f))
    return out


def _stale(obj: str, src: str, headers) -> bool:
    if not os.path.exists(obj):
        return True
    t = os.path.getmtime(obj)
    return any(os.path.getmtime(p) > t for p in [src, *headers, __file__])


def _compile(cmd, log_path=None):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if log_path is not None:
        with open(log_path, "w") as f:
            f.write(r.stdout + r.stderr)
    if r.returncode != 0:
        raise RuntimeError("compile failed:\n" + " ".join(cmd) + "\n" + r.stdout + r.stderr)
    return r.stdout + r.stderr


def _binding_command(home: str, out: str):
    """g++ command of the binding that reads torch tensors in C++, and the
    file whose age says which torch it was built against."""
    import sysconfig

    import torch

    base = os.path.dirname(torch.__file__)
    inc = [os.path.join(base, "include"), os.path.join(base, "include", "torch", "csrc", "api", "include"),
           os.path.join(home, "include"), sysconfig.get_paths()["include"], INCLUDE]
    lib = os.path.join(base, "lib")
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}"]
    for p in inc:
        cmd += ["-isystem" if p != INCLUDE else "-I", p]
    cmd += [BINDING_SOURCE, "-o", out, f"-L{lib}", f"-Wl,-rpath,{lib}", "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch",
            "-ltorch_python"]
    return cmd, os.path.join(base, "version.py")


def build(force: bool = False, verbose: bool = False) -> str:
    home = cuda_home()
    nvcc = os.path.join(home, "bin", "nvcc")
    os.makedirs(BUILD, exist_ok=True)
    headers = _headers()
    common = ["-O3", "-std=c++17", "-I", INCLUDE, "-I", CSRC, "-Xcompiler", "-fPIC"]
    jobs = []
    objs = []
    for src in CU_SOURCES:
        s = os.path.join(CSRC, src)
        o = os.path.join(BUILD, src + ".o")
        objs.append(o)
        if force or _stale(o, s, headers):
            cmd = [nvcc, *ARCH, "-lineinfo", "-Xptxas", "-v", *common, "-c", s, "-o", o]
            jobs.append((cmd, os.path.join(BUILD, src + ".ptxas.log")))
    for src in CPP_SOURCES:
        s = os.path.join(CSRC, src)
        o = os.path.join(BUILD, src + ".o")
        objs.append(o)
        if force or _stale(o, s, headers):
            cmd = [nvcc, *ARCH, *common, "-x", "c++", "-c", s, "-o", o]
            jobs.append((cmd, None))
    tmp_binding = BINDING + f".tmp{os.getpid()}"
    command, torch_version = _binding_command(home, tmp_binding)
    bind = force or _stale(BINDING, BINDING_SOURCE, [os.path.join(INCLUDE, "mdcn.h"), torch_version])
    bound = None
    if jobs or bind:
        with cf.ThreadPoolExecutor(max_workers=max(1, min(len(jobs) + bind, os.cpu_count() or 1))) as ex:
            futs = [ex.submit(_compile, c, l) for c, l in jobs]
            if bind:  # what goes wrong with it is raised below, once the library is there
                bound = ex.submit(_compile, command)
            for f in futs:
                out = f.result()
                if verbose and out:
                    print(out)
        with open(os.path.join(BUILD, "ptxas.log"), "w") as f:
            for src in CU_SOURCES:
                p = os.path.join(BUILD, src + ".ptxas.log")
                if os.path.exists(p):
                    f.write(open(p).read())
    if force or jobs or not os.path.exists(LIB) or any(os.path.getmtime(o) > os.path.getmtime(LIB) for o in objs):
        tmp = LIB + f".tmp{os.getpid()}"
        lib64 = os.path.join(home, "lib64")
        cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *objs, "-lcublas", "-Xlinker", f"-rpath,{lib64}"]
        _compile(cmd)
        os.replace(tmp, LIB)
    if bound is not None:
        bound.result()
        os.replace(tmp_binding, BINDING)
    return LIB


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("-v", "--verbose", action="store_true")
    a = ap.parse_args(argv)
    print(build(force=a.force, verbose=a.verbose))


if __name__ == "__main__":
    sys.exit(main())
