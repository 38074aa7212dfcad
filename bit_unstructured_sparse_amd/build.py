"""Builds libbitmap_spmm.so (and the streaming-read probe libbsp_probe.so)
in this directory with hipcc for gfx950, and the binding's native steps
(_binding.so) with the host compiler against PyTorch's headers.

    python -m bit_unstructured_sparse_amd.build

One shared library holds the host encoders (encode.cpp, encode_union.cpp,
encode_cbc.cpp, encode_int8.cpp) and every HIP kernel
(spmm.hip with its kernels_*.hip includes, kv_cache.hip, attention_tree.hip, kv_pages.hip,
qk_heads.hip, quantize_tokens.hip, gemm_w8a8.hip). The probe (probe_read.hip) is a
measurement aid the benchmark loads; the SpMM library does not contain it.
Packed-fp32 VALU forms are switched off for the device pass; hipcc's host
pass warns that it does not know that feature, which is harmless.
"""
from __future__ import annotations

import importlib.util
import os
import subprocess
import sys
import sysconfig
import tempfile
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libbitmap_spmm.so")
PROBE_LIB = os.path.join(HERE, "libbsp_probe.so")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
ARCH = "gfx950"

SOURCES = [os.path.join(CSRC, "spmm.hip"), os.path.join(CSRC, "encode.cpp"), os.path.join(CSRC, "encode_union.cpp"),
           os.path.join(CSRC, "encode_cbc.cpp"), os.path.join(CSRC, "encode_int8.cpp"),
           os.path.join(CSRC, "kv_cache.hip"), os.path.join(CSRC, "attention_tree.hip"),
           os.path.join(CSRC, "kv_pages.hip"), os.path.join(CSRC, "qk_heads.hip"),
           os.path.join(CSRC, "quantize_tokens.hip"), os.path.join(CSRC, "gemm_w8a8.hip")]
PROBE_SOURCES = [os.path.join(CSRC, "probe_read.hip")]


# The steps that the binding's calls repeat, natively; without PyTorch there is nothing to build them for.
BINDING = os.path.join(HERE, "_binding.so")
BINDING_SOURCES = [os.path.join(CSRC, "binding.cpp")]


def binding_command(out: str):
    """The host compiler's command, or None without PyTorch."""
    spec = importlib.util.find_spec("torch")
    if spec is None:
        return None
    torch = spec.submodule_search_locations[0]
    rocm = os.path.dirname(os.path.dirname(HIPCC))
    return [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", "-D__HIP_PLATFORM_AMD__",
            "-DUSE_ROCM", "-I", os.path.join(ROOT, "include"), "-isystem", os.path.join(torch, "include"),
            "-isystem", os.path.join(torch, "include", "torch", "csrc", "api", "include"),
            "-isystem", sysconfig.get_paths()["include"], "-isystem", os.path.join(rocm, "include"),
            *BINDING_SOURCES, "-o", out, "-L", os.path.join(torch, "lib"), "-ltorch_python", "-ltorch", "-ltorch_cpu",
            "-ltorch_hip", "-lc10", "-lc10_hip"]


FLAGS = [f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC", "-I", os.path.join(ROOT, "include"), "-I", CSRC,
         "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops", "-Wall", "-Wno-unused-function"]


def _run(cmd, verbose: bool) -> None:
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    noise = "'-packed-fp32-ops' is not a recognized feature"
    msgs = [ln for ln in (r.stdout + r.stderr).splitlines() if noise not in ln]
    if r.returncode != 0:
        raise RuntimeError(f"{os.path.basename(cmd[0])} failed:\n" + "\n".join(msgs))
    if verbose and msgs:
        print("\n".join(msgs), flush=True)


def _library(out: str, sources, pool, verbose: bool) -> str:
    """The sources compiled side by side and linked; `out` is replaced at the end."""
    tmp = out + f".tmp{os.getpid()}"
    with tempfile.TemporaryDirectory() as folder:
        objects = [os.path.join(folder, os.path.basename(s) + ".o") for s in sources]
        list(pool.map(lambda so: _run([HIPCC, *FLAGS, "-c", so[0], "-o", so[1]], verbose), zip(sources, objects)))
        _run([HIPCC, f"--offload-arch={ARCH}", "-fPIC", "-shared", *objects, "-o", tmp, "-lpthread"], verbose)
    os.replace(tmp, out)
    return out


def _binding(verbose: bool) -> None:
    """The native module, where it can be built. Where it cannot (no host compiler, no headers or GPU libraries of
    PyTorch) that is reported, and the binding's Python functions do its work: one of other sources must not stay."""
    tmp = BINDING + f".tmp{os.getpid()}"
    cmd = binding_command(tmp)
    if cmd is None:
        return
    try:
        _run(cmd, verbose)
        os.replace(tmp, BINDING)
    except (RuntimeError, OSError) as e:
        for left in (tmp, BINDING):
            if os.path.exists(left):
                os.remove(left)
        print(f"{os.path.basename(BINDING)} not built, calls go through ctypes: {e}", file=sys.stderr, flush=True)


def build(verbose: bool = False) -> str:
    with ThreadPoolExecutor(min(8, int(os.environ.get("MAX_JOBS", 8)))) as pool, ThreadPoolExecutor(1) as other:
        binding = other.submit(_binding, verbose)
        _library(PROBE_LIB, PROBE_SOURCES, pool, verbose)
        _library(LIB, SOURCES, pool, verbose)
        binding.result()
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
