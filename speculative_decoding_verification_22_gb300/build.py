"""Builds ``libspec_verify.so`` in-tree for sm_103a with nvcc, and the compiled
Python binding of the target-layer operators beside it.

Each CUDA translation unit is compiled in parallel into ``_build/`` and
linked with the static CUDA runtime, so the library loads on machines
without a GPU (for symbol checks) and needs only the driver at run time.
The library does not need the binding: it is linked first, and stands where
the binding fails to build or torch is missing or has no CUDA.
"""
from __future__ import annotations

import concurrent.futures
import os
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libspec_verify.so")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
SOURCES = ["sv_api.cu", "sv_lmhead_tc.cu", "sv_lmhead_simt.cu", "sv_tail.cu", "sv_noalloc.cu",
           "sv_trunc.cu",
           "sv_ngram.cu",
           "sv_target_api.cu", "sv_norm.cu", "sv_rope.cu", "sv_matmul8.cu", "sv_attn.cu",
           "sv_attn_tc.cu"]
HEADERS = ["sv_internal.cuh", "sv_kernels.h", "sv_target.cuh", "sv_attn.cuh",
           "sv_tmem.cuh"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
         "--expt-relaxed-constexpr", "-I", INCLUDE]


BIND_SRC = os.path.join(CSRC, "sv_bind.cpp")
BIND = os.path.join(HERE, "_target_bind.so")


def _bind_commands():
    """(compile, link, object) of the binding for the torch that is installed;
    None where there is none with CUDA, and nothing to bind."""
    try:
        import torch
    except ImportError:
        return None
    if torch.version.cuda is None:
        return None
    t = os.path.dirname(torch.__file__)
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    obj = os.path.join(BUILD, f"sv_bind.{torch.__version__}.o")
    inc = [os.path.join(t, "include"),
           os.path.join(t, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], os.path.join(cuda, "include"), INCLUDE]
    flags = ["-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden",
             f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"]
    compile_ = ["g++", *flags, *[x for i in inc for x in ("-I", i)], "-c", BIND_SRC, "-o", obj]
    lib = os.path.join(t, "lib")
    link = ["g++", "-shared", obj, "-L", lib, "-lc10", "-lc10_cuda", "-ltorch_cpu",
            "-ltorch_cuda", "-ltorch_python", "-L", HERE, "-l:libspec_verify.so",
            "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{lib}"]
    return compile_, link, obj


def _nvcc():
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    path = os.path.join(cuda, "bin", "nvcc")
    return path if os.path.exists(path) else "nvcc"


def _stale(out, deps):
    if not os.path.exists(out):
        return True
    t = os.path.getmtime(out)
    return any(os.path.getmtime(p) > t for p in deps)


def build(force: bool = False, ptxas_verbose: bool = False, verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()
    hdrs = [os.path.join(CSRC, h) for h in HEADERS] + [
        os.path.join(INCLUDE, h) for h in ("spec_verify.h", "spec_target.h")]
    jobs = []
    objs = []
    for src in SOURCES:
        s = os.path.join(CSRC, src)
        o = os.path.join(BUILD, src.replace(".cu", ".o"))
        objs.append(o)
        if force or _stale(o, [s] + hdrs):
            cmd = [nvcc, *ARCH, *FLAGS, "-c", s, "-o", o]
            if ptxas_verbose:
                cmd.append("-Xptxas=-v")
            jobs.append(cmd)

    bind = _bind_commands()
    bind_job = bind is not None and (force or _stale(bind[2], [BIND_SRC] + hdrs))
    if bind_job:
        jobs.insert(0, bind[0])

    def run(cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        return cmd, r

    failed = bind_failed = None
    if jobs:
        with concurrent.futures.ThreadPoolExecutor(max_workers=len(jobs)) as ex:
            for i, (cmd, r) in enumerate(ex.map(run, jobs)):
                if verbose or ptxas_verbose or r.returncode != 0:
                    sys.stderr.write(r.stdout + r.stderr)
                if r.returncode != 0:
                    what = f"compilation failed: {' '.join(cmd)}"
                    if bind_job and i == 0:
                        bind_failed = what
                    else:
                        failed = failed or what
    if failed:
        raise RuntimeError(failed)
    if force or _stale(LIB, objs):
        tmp = LIB + f".tmp{os.getpid()}"
        cmd = [nvcc, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs,
               "-ldl", "-lpthread", "-lrt"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            sys.stderr.write(r.stdout + r.stderr)
            raise RuntimeError("link failed")
        os.replace(tmp, LIB)
    if bind is None:
        sys.stderr.write("no torch with CUDA: the Python binding of the target-layer "
                         "operators is not built\n")
        return LIB
    if bind_failed:
        raise RuntimeError(bind_failed)
    _, bind_link, bind_obj = bind
    if force or _stale(BIND, [bind_obj, LIB]):
        tmp = BIND + f".tmp{os.getpid()}"
        r = subprocess.run([*bind_link, "-o", tmp], capture_output=True, text=True)
        if r.returncode != 0:
            sys.stderr.write(r.stdout + r.stderr)
            raise RuntimeError("link of the binding failed")
        os.replace(tmp, BIND)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, ptxas_verbose="-v" in sys.argv, verbose=True)
