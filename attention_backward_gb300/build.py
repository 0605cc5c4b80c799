"""Builds the CUDA library ``_build/libattn_bwd.so`` for sm_103a with nvcc, and
``_build/libattn_torch.so``, Python functions on torch tensors over some of its entry points.

Each translation unit is compiled in parallel, then linked into one shared
library with the CUDA runtime linked statically, so the library loads on a
machine without a GPU (the driver is looked up only when a call needs it).
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(BUILD, "libattn_bwd.so")
TORCH_LIB = os.path.join(BUILD, "libattn_torch.so")
TORCH_SOURCE = "torch_latent.cpp"
SOURCES = ["api.cu", "preprocess.cu", "dense_bwd.cu", "dense128_bwd.cu", "dense_fwd.cu", "sparse_bwd.cu", "noalloc.cu", "host_pipeline.cu",
           "kv_api.cu", "kv_cache.cu", "kv_decode.cu", "kv_prompt.cu", "kv_join.cu",
           "rope.cu", "latent_api.cu", "latent_write.cu", "latent_attn.cu", "latent_join.cu", "latent_fwd.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
         "--expt-relaxed-constexpr", "-I", os.path.join(ROOT, "include"), "-I", CSRC]


def nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _stale(obj: str, src: str) -> bool:
    if not os.path.exists(obj):
        return True
    t = os.path.getmtime(obj)
    deps = [src] + [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    inc = os.path.join(ROOT, "include")
    deps += [os.path.join(inc, f) for f in os.listdir(inc)]
    return any(os.path.getmtime(d) > t for d in deps)


def _torch_flags(cc: str) -> tuple:
    """Flags that compile and link against the torch of this interpreter."""
    import sysconfig

    import torch

    at = os.path.dirname(torch.__file__)
    include = [os.path.join(at, "include"), os.path.join(at, "include", "torch", "csrc", "api", "include"),
               os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(cc))), "include"), os.path.join(ROOT, "include"),
               sysconfig.get_paths()["include"]]
    return (["-O2", "-std=c++17", "-fPIC", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
             *(f"-I{i}" for i in include)],
            [f"-L{os.path.join(at, 'lib')}", "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch", "-ltorch_python"])


def _newer(lib: str, objs) -> bool:
    """Whether ``lib`` has to be linked again.  By the files' times and not by what this run
    compiled, so that a build that failed half way is taken up by the next one."""
    return not os.path.exists(lib) or any(os.path.getmtime(o) > os.path.getmtime(lib) for o in objs)


def build(verbose: bool = False, force: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()
    objs, jobs = [], []
    for s in SOURCES:
        src = os.path.join(CSRC, s)
        obj = os.path.join(BUILD, s.replace(".cu", ".o"))
        objs.append(obj)
        if force or _stale(obj, src):
            jobs.append((obj, [cc, *ARCH, *FLAGS, "-c", src] + (["-Xptxas", "-v"] if verbose else [])))

    def run(job):  # a file takes its name when it is whole
        to, cmd = job
        tmp = to + ".tmp"
        r = subprocess.run([*cmd, "-o", tmp], capture_output=True, text=True)
        if r.returncode == 0:
            os.replace(tmp, to)
        return cmd, r

    def check(cmd, r, what):
        if verbose or r.returncode:
            sys.stderr.write(r.stdout + r.stderr)
        if r.returncode:
            raise RuntimeError(f"{what} failed: {' '.join(cmd)}")

    with ThreadPoolExecutor(len(jobs) + 1) as ex:
        extension = ex.submit(_compile_extension, cc, force, run, check)
        for cmd, r in ex.map(run, jobs):
            check(cmd, r, "compiler")
    if force or _newer(LIB, objs):
        check(*run((LIB, [cc, *ARCH, "-shared", *objs, "-cudart", "static"])), "link")
    # (the library needs neither torch nor Python's headers and is there whatever the extension lacks)
    obj, link = extension.result()
    if force or _newer(TORCH_LIB, [obj]):
        check(*run((TORCH_LIB, link)), "link")
    return LIB


def _compile_extension(cc: str, force: bool, run, check) -> tuple:
    """Its object, and the command that links it."""
    cxx = shutil.which("g++") or "g++"
    compile_flags, link_flags = _torch_flags(cc)
    obj, src = os.path.join(BUILD, "torch_latent.o"), os.path.join(CSRC, TORCH_SOURCE)
    # its ABI is this interpreter's and this torch's: what an object was made for stands beside it
    import torch

    stamp, made_for = obj + ".for", "\n".join([torch.__version__, sys.version, *compile_flags, *link_flags])
    if force or _stale(obj, src) or not os.path.exists(stamp) or open(stamp).read() != made_for:
        if os.path.exists(stamp):
            os.remove(stamp)
        check(*run((obj, [cxx, *compile_flags, "-c", src])), "compiler")
        with open(stamp, "w") as f:
            f.write(made_for)
    return obj, [cxx, "-shared", obj, f"-L{BUILD}", f"-l:{os.path.basename(LIB)}", "-Wl,-rpath,$ORIGIN", *link_flags]


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv, force="-f" in sys.argv))
