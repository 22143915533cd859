"""Builds libmxmlp.so (the C-ABI library) in-tree with nvcc for sm_103a.

Each .cu file is compiled to an object in parallel, then the objects are
linked into ``block_scaled_mlp_gb300/libmxmlp.so`` (static CUDA runtime, no
libcuda link: the driver entry point for tensor maps is looked up at run
time, so the library also loads on machines without a GPU driver).  Beside it
``_binding.so``, the Python binding of the operators whose calls are short
(csrc/binding.cpp, compiled against the installed torch's headers, and again
when another torch is installed).  Where that does not compile the library is
built all the same, with a warning; the calls that need the binding then raise.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libmxmlp.so")
BINDING = os.path.join(HERE, "_binding.so")
SOURCES = ["api.cu", "quant.cu", "swiglu.cu", "gemm.cu", "dispatch.cu", "norm.cu", "ckpt8.cu",
           "ragged.cu", "route.cu", "combine.cu", "fp8block.cu", "fp8mm.cu", "ops.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
         "--expt-relaxed-constexpr"]


def _nvcc() -> str:
    cand = [os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc"), shutil.which("nvcc")]
    for c in cand:
        if c and os.path.exists(c):
            return c
    raise RuntimeError("nvcc not found (set CUDA_HOME)")


def _stale(obj: str, deps) -> bool:
    if not os.path.exists(obj):
        return True
    t = os.path.getmtime(obj)
    return any(os.path.getmtime(d) > t for d in deps)


def _torch_flags():
    """Compile and link flags of a Python extension on the installed torch."""
    import sysconfig

    import torch

    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(_nvcc()))
    inc = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
           os.path.join(cuda, "include"), sysconfig.get_paths()["include"]]
    abi = f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}"
    libs = [f"-L{os.path.join(root, 'lib')}", "-ltorch_python", "-ltorch_cuda", "-ltorch_cpu", "-lc10_cuda", "-lc10"]
    return [abi, *("-I" + i for i in inc)], libs


def _torch_key() -> str:
    """What a compiled binding depends on besides its sources."""
    import torch

    return f"{sys.implementation.cache_tag} torch {torch.__version__} {os.path.dirname(torch.__file__)}"


def build(verbose: bool = False, force: bool = False, extra_flags=None) -> str:
    nvcc = _nvcc()
    os.makedirs(BUILD, exist_ok=True)
    headers = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    headers.append(os.path.join(os.path.dirname(HERE), "include", "mxmlp.h"))
    extra = list(extra_flags or [])

    def compile_one(src):
        s = os.path.join(CSRC, src)
        o = os.path.join(BUILD, src.replace(".cu", ".o"))
        if not force and not _stale(o, [s] + headers):
            return o, None
        cmd = [nvcc, *ARCH, *FLAGS, *extra, "-c", s, "-o", o]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
        return o, r.stdout + r.stderr

    def run(cmd, what):
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"{what} failed:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")

    binding_src, binding_obj = os.path.join(CSRC, "binding.cpp"), os.path.join(BUILD, "binding.o")
    key_file, key = os.path.join(BUILD, "binding.key"), _torch_key()

    def compile_binding():
        old = open(key_file).read() if os.path.exists(key_file) else None
        if force or old != key or _stale(binding_obj, [binding_src, headers[-1]]):
            if os.path.exists(key_file):
                os.remove(key_file)
            run(["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", *_torch_flags()[0], "-c", binding_src, "-o",
                 binding_obj], "g++ for binding.cpp")
            with open(key_file, "w") as f:
                f.write(key)
            return True
        return False

    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        binding = ex.submit(compile_binding)
        results = list(ex.map(compile_one, SOURCES))
    objs = [o for o, _ in results]
    if verbose:
        for _, log in results:
            if log and log.strip():
                print(log, file=sys.stderr)
    # what was compiled is linked again, even where file times are too coarse to show it
    if force or any(log is not None for _, log in results) or _stale(LIB, objs):
        cmd = [nvcc, *ARCH, "-shared", "-Xcompiler", "-fPIC", "-o", LIB, *objs]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    try:
        if binding.result() or force or _stale(BINDING, [binding_obj]):
            run(["g++", "-shared", "-o", BINDING, binding_obj, f"-L{HERE}", "-l:libmxmlp.so", "-Wl,-rpath,$ORIGIN",
                 *_torch_flags()[1]], "link of the binding")
    except (RuntimeError, OSError) as e:
        if os.path.exists(BINDING):  # one of other sources or another torch
            os.remove(BINDING)
        print(f"warning: {BINDING} is not built, the operators around the MLP will raise\n{e}", file=sys.stderr)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True, force="--force" in sys.argv))
