"""Build the CUDA library ``libattn.so`` in-tree with nvcc for sm_103a.

The translation units (the host ABI, the host-buffer pipeline, the attention
block's GEMM and LayerNorm, the families of attention-kernel variants, the
paged cache's append and attention, the backward pass, checkpoints, rotary axes) are compiled in parallel to objects under
``_build/`` and linked into one shared library; one -gencode, no cmake. Beside
it stands ``_binding.so``, a small Python module over that library for the calls
of a decode step (g++, against PyTorch's headers). The results sit next to this
file and are git-ignored.
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
ROOT = os.path.dirname(HERE)
LIBRARY = os.path.join(HERE, "libattn.so")
BINDING = os.path.join(HERE, "_binding.so")
OBJDIR = os.path.join(HERE, "_build")
SOURCES = [os.path.join(CSRC, f) for f in
           ("attn_api.cu", "attn_host.cu", "block_kernels.cu", "fwd_bf16.cu", "fwd_f16.cu", "fwd_rope_bf16.cu",
            "fwd_rope_f16.cu", "fwd_pack_bf16.cu", "fwd_pack_f16.cu", "fwd_window_bf16.cu",
            "fwd_window_f16.cu", "paged_api.cu", "paged_append.cu", "paged_gather.cu",
            "paged_attn_bf16.cu", "paged_attn_f16.cu", "paged_attn_e4m3.cu", "bwd_api.cu", "bwd_small.cu",
            "bwd_bf16_d64.cu", "bwd_bf16_d128.cu", "bwd_f16_d64.cu", "bwd_f16_d128.cu",
            "checkpoint.cu", "rope_axes.cu")]
DEPENDS = SOURCES + [os.path.join(CSRC, f) for f in
                     ("attn_kernel.cuh", "ptx.cuh", "attn_launch.h", "attn_fwd_inst.cuh", "block_params.h",
                      "gemm_kernel.cuh", "early_launch.h", "paged_params.h", "paged_attn.cuh", "bwd_params.h",
                      "bwd_kernel.cuh", "bwd_inst.cuh", "checkpoint_params.h", "e4m3.cuh")] + [
    os.path.join(ROOT, "include", "attn.h")]
BINDING_SOURCE = os.path.join(CSRC, "binding.cpp")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = [*ARCH, "-lineinfo", "-O3", "-std=c++17", "-Xcompiler", "-fPIC"]


def nvcc_path() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libattn.so")


def up_to_date(output: str = LIBRARY, depends=DEPENDS) -> bool:
    if not os.path.exists(output):
        return False
    t = os.path.getmtime(output)
    return all(os.path.getmtime(d) <= t for d in depends)


def build_binding(force: bool = False, library: str = LIBRARY, output: str = BINDING) -> str:
    """The Python module of the per-step calls, linked against the library that stands beside it."""
    torch = importlib.util.find_spec("torch").submodule_search_locations[0]
    depends = [BINDING_SOURCE, os.path.join(ROOT, "include", "attn.h"), os.path.join(torch, "version.py")]
    if not force and up_to_date(output, depends):
        return output
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc_path())))
    subprocess.run(["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-I", os.path.join(ROOT, "include"),
                    "-I", sysconfig.get_paths()["include"], "-I", os.path.join(torch, "include"),
                    "-I", os.path.join(torch, "include", "torch", "csrc", "api", "include"),
                    "-I", os.path.join(cuda, "include"), "-o", output + ".tmp", BINDING_SOURCE,
                    "-L", os.path.join(torch, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda",
                    "-L", os.path.dirname(library), "-l:" + os.path.basename(library), "-Wl,-rpath,$ORIGIN"], check=True)
    os.replace(output + ".tmp", output)
    return output


def build(force: bool = False, output: str = LIBRARY, verbose: bool = False) -> str:
    if force or not up_to_date(output):
        build_library(output, verbose)
    if output == LIBRARY:
        build_binding(force)
    return output


def build_library(output: str, verbose: bool) -> None:
    nvcc = nvcc_path()
    os.makedirs(OBJDIR, exist_ok=True)
    include = ["-I", os.path.join(ROOT, "include")]

    def compile_one(src: str) -> str:
        obj = os.path.join(OBJDIR, os.path.splitext(os.path.basename(src))[0] + ".o")
        cmd = [nvcc, *FLAGS, *include, "-c", "-o", obj, src]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        subprocess.run(cmd, check=True)
        return obj

    with ThreadPoolExecutor(max_workers=min(len(SOURCES), os.cpu_count() or 1)) as pool:
        objects = list(pool.map(compile_one, SOURCES))
    subprocess.run([nvcc, *ARCH, "-shared", "-o", output + ".tmp", *objects], check=True)
    os.replace(output + ".tmp", output)


if __name__ == "__main__":  # pragma: no cover
    print(build(force=True, verbose=True))
