"""Compile the HIP library ``libnf4.so`` for gfx950, in-tree, the host-CPU pass
``libnf4cpu.so`` and the Python calls' plain case ``_calls.so`` beside it.

hipcc cross-compiles without a GPU, one process per source (the matmul files
take about a minute each).  Flags: no fast-math and no FMA
contraction (the codec's fp32 steps are specified as separately rounded
operations), packed fp32 instructions off, fp32 denormals kept (the default).
"""
from __future__ import annotations

import os
import subprocess
import sys
import tempfile
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB_PATH = os.path.join(PKG, "libnf4.so")
CPU_LIB_PATH = os.path.join(PKG, "libnf4cpu.so")
CALLS_PATH = os.path.join(PKG, "_calls.so")
CPU_SOURCES = [os.path.join("cpu", "nf4_cpu.cpp")]
SOURCES = ["k_gemm.hip", "k_linear_back.hip", "k_linear.hip", "k_codec.hip", "k_lora.hip", "k_variants.hip",
           "k_norm.hip", "k_mx4_mm.hip", "k_mx4_mm4.hip", "k_mx4_few.hip", "k_mx4.hip", "k_select.hip",
           "nf4_scratch.hip", "nf4_api.cpp", "mx4_api.cpp"]
ARCH = os.environ.get("NF4_OFFLOAD_ARCH", "gfx950")


def compile_command(source: str, out: str) -> list:
    return ["hipcc", f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC",
            "-ffp-contract=off", "-fno-fast-math",
            "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
            "-Wall", "-Wno-unused-command-line-argument",
            "-I", os.path.join(ROOT, "include"), "-I", CSRC,
            "-c", "-o", out, os.path.join(CSRC, source)]


def link_command(objects: list, out: str = LIB_PATH) -> list:
    return ["hipcc", f"--offload-arch={ARCH}", "-shared", "-fPIC", "-o", out, *objects]


def cpu_command(out: str = CPU_LIB_PATH) -> list:
    """The host-CPU pass (OpenMP, AVX2 baseline with an AVX-512 tile path chosen at run time,
    no FMA contraction)."""
    return ["g++", "-O3", "-march=x86-64-v3", "-std=c++17", "-fPIC", "-shared", "-fopenmp",
            "-ffp-contract=off", "-fno-fast-math", "-Wall",
            "-I", os.path.join(ROOT, "include"), "-I", CSRC,
            "-o", out, *[os.path.join(PKG, s) for s in CPU_SOURCES]]


def build_cpu(verbose: bool = False) -> str:
    tmp = CPU_LIB_PATH + ".tmp"
    cmd = cpu_command(tmp)
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed ({r.returncode}):\n{r.stderr}")
    os.replace(tmp, CPU_LIB_PATH)
    return CPU_LIB_PATH


def calls_command(out: str = CALLS_PATH) -> list:
    """The Python calls' plain case (a CPython module against torch's C++ tensors)."""
    import sysconfig

    import torch
    t = os.path.dirname(torch.__file__)
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", "-Wall", "-Wno-attributes",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
            "-I", os.path.join(ROOT, "include"), "-isystem", os.path.join(t, "include"),
            "-isystem", sysconfig.get_paths()["include"], "-o", out, os.path.join(CSRC, "py_calls.cpp"),
            "-L", os.path.join(t, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", f"-Wl,-rpath,{os.path.join(t, 'lib')}"]


def build_calls(verbose: bool = False) -> str:
    tmp = CALLS_PATH + ".tmp"
    cmd = calls_command(tmp)
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed ({r.returncode}):\n{r.stderr}")
    os.replace(tmp, CALLS_PATH)
    return CALLS_PATH


def build_calls_if_possible(verbose: bool = False) -> str | None:
    """build_calls where g++, torch's and Python's C++ headers are there.  Without the module
    every call works (Python checks it instead), so a failure is reported and no error; a
    module of an older source does not stay."""
    try:
        return build_calls(verbose)
    except (RuntimeError, OSError, ImportError) as e:
        if os.path.exists(CALLS_PATH):
            os.remove(CALLS_PATH)
        print(f"warning: {os.path.basename(CALLS_PATH)} was not built, small calls from Python will be slower: {e}",
              file=sys.stderr, flush=True)
        return None


def _hipcc(cmd: list, verbose: bool) -> None:
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    # the host pass does not know the packed-fp32 feature and says so; harmless
    err = "\n".join(l for l in r.stderr.splitlines()
                    if "packed-fp32-ops" not in l and l.strip())
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed ({r.returncode}):\n{err}")
    if err and verbose:
        print(err, file=sys.stderr)


def build(verbose: bool = False) -> str:
    tmp = LIB_PATH + ".tmp"
    with tempfile.TemporaryDirectory() as d:
        objects = [os.path.join(d, s + ".o") for s in SOURCES]
        with ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as pool:
            for f in [pool.submit(_hipcc, compile_command(s, o), verbose) for s, o in zip(SOURCES, objects)]:
                f.result()
        _hipcc(link_command(objects, tmp), verbose)
    os.replace(tmp, LIB_PATH)
    return LIB_PATH


if __name__ == "__main__":
    print(build(verbose=True))
    print(build_cpu(verbose=True))
    print(build_calls_if_possible(verbose=True))
