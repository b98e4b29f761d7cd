"""Build libnvfp4fc2.so and the Python module of the MXFP4 functions in-tree
for sm_103a (nvcc, g++, no cmake).

Steps: generate the BF16 silu table header, compile each .cu in parallel
with ``-gencode arch=compute_103a,code=sm_103a -lineinfo -O3`` (IEEE
division and square root, no flush-to-zero, no fast math), link a shared
library with the CUDA runtime linked statically; g++ compiles binding.cpp
against PyTorch's headers.  Output:
``diffusion_transformer_mlp_gb300/_build/libnvfp4fc2.so`` and ``_mxfp4.so``.
"""
from __future__ import annotations

import concurrent.futures
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
GEN = os.path.join(BUILD, "gen")
LIB = os.path.join(BUILD, "libnvfp4fc2.so")
BINDING = os.path.join(BUILD, "_mxfp4.so")
SOURCES = ["api.cu", "quant.cu", "gemm.cu", "mma_peak.cu", "tc_read.cu", "noalloc.cu",
           "mx_quant.cu", "mx_cache.cu", "mx_rows.cu", "mx_linear.cu", "mx_attn.cu", "mx_attn_stream.cu",
           "mx_attn_chunk.cu", "mx_attn_combine.cu", "mx_attn_shared.cu", "mx_rotary.cu", "mx_pages.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + ["-lineinfo", "-O3", "-std=c++17", "-Xcompiler", "-fPIC", "-ftz=false", "-prec-div=true",
                     "-prec-sqrt=true", "-fmad=true", "-Xptxas", "-v"]


def nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found")
    return cand


def _binding_job():
    """Command that makes the Python module."""
    import sysconfig

    import torch
    t = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    inc = [INCLUDE, os.path.join(t, "include"), os.path.join(t, "include", "torch", "csrc", "api", "include"),
           os.path.join(cuda, "include"), sysconfig.get_paths()["include"]]
    cmd = (["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"] + [a for i in inc for a in ("-I", i)]
           + [os.path.join(CSRC, "binding.cpp"), "-o", BINDING + f".tmp{os.getpid()}", "-L", os.path.join(t, "lib"),
              "-lc10", "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python", "-lc10_cuda"])
    return cmd


def _torch_stamp() -> str:
    import torch
    return f"{torch.__version__} {sys.implementation.cache_tag}"


def binding_is_current() -> bool:
    """The Python module exists and was compiled against this PyTorch and Python,
    whose binary interfaces it uses."""
    try:
        with open(BINDING + ".torch") as f:
            return os.path.exists(BINDING) and f.read() == _torch_stamp()
    except OSError:
        return False


def _newer(target: str, deps: list[str]) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _headers() -> list[str]:
    hs = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    hs += [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE) if f.endswith(".h")]
    return hs


def build(verbose: bool = False, force: bool = False) -> str:
    os.makedirs(GEN, exist_ok=True)
    table = os.path.join(GEN, "silu_table_full.inc")
    gen = os.path.join(CSRC, "gen_silu_table.py")
    if force or _newer(table, [gen]):
        subprocess.check_call([sys.executable, gen, table])
    deps = _headers() + [table]
    objs, jobs = [], []
    binding = force or not binding_is_current() or _newer(BINDING, [os.path.join(CSRC, "binding.cpp")] + deps)
    if binding:
        jobs.append(("binding.cpp", _binding_job()))
    for src in SOURCES:
        s = os.path.join(CSRC, src)
        o = os.path.join(BUILD, src.replace(".cu", ".o"))
        objs.append(o)
        if force or _newer(o, [s] + deps):
            cmd = [nvcc()] + NVCC_FLAGS + ["-I", INCLUDE, "-I", CSRC, "-I", GEN, "-c", s, "-o", o]
            jobs.append((src, cmd))

    def run(job):
        src, cmd = job
        r = subprocess.run(cmd, capture_output=True, text=True)
        return src, r

    with concurrent.futures.ThreadPoolExecutor(max_workers=max(1, len(jobs))) as ex:
        for src, r in ex.map(run, jobs):
            log = r.stdout + r.stderr
            if r.returncode != 0:
                raise RuntimeError(f"nvcc failed on {src}:\n{log}")
            with open(os.path.join(BUILD, src + ".ptxas.txt"), "w") as f:
                f.write(log)
            if verbose:
                print(log)
    if binding:
        os.replace(BINDING + f".tmp{os.getpid()}", BINDING)
        with open(BINDING + ".torch", "w") as f:
            f.write(_torch_stamp())
    if force or jobs or not os.path.exists(LIB):
        tmp = LIB + f".tmp{os.getpid()}"
        subprocess.check_call([nvcc()] + ARCH + ["-shared", "-o", tmp] + objs)
        os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv, force="-f" in sys.argv))
