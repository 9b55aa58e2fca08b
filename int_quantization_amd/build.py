"""Build libiq.so in-tree with hipcc for gfx950."""
from __future__ import annotations

import os
import subprocess
import tempfile
from concurrent.futures import ThreadPoolExecutor

_HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(_HERE)
SOURCES = [os.path.join(_HERE, "csrc", name) for name in
           ("iq_kernels.hip", "iq_api.cpp", "iq_norm.hip", "iq_packed.hip", "iq_gated.hip", "iq_ffn_api.cpp", "iq_cache.hip", "iq_attend.hip",
            "iq_attn_api.cpp")]
OUT = os.path.join(_HERE, "libiq.so")
BENCH_SOURCES = [os.path.join(_HERE, "csrc", "bench_copy.hip")]
BENCH_OUT = os.path.join(_HERE, "libiq_bench.so")
FAST_SOURCE = os.path.join(_HERE, "csrc", "iq_fast.cpp")
FAST_OUT = os.path.join(_HERE, "_fast.so")

HIPCC_FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC",
    # no FMA contraction: x - s*q and the statistics must round as written
    "-ffp-contract=off",
    # no packed FP32 (v_pk_fma_f32 / v_pk_mul_f32 / v_pk_add_f32) in device code
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall",
]


def _run(cmd, verbose):
    r = subprocess.run(cmd, capture_output=True, text=True)
    noise = "'-packed-fp32-ops' is not a recognized feature"
    msgs = [ln for ln in (r.stdout + r.stderr).splitlines() if noise not in ln]
    if r.returncode != 0:
        raise RuntimeError("hipcc failed:\n" + "\n".join(msgs))
    if verbose and msgs:
        print("\n".join(msgs))


def _hipcc(sources, out, verbose):
    """Compile every source to an object of its own, a few at a time, and link them."""
    hipcc = [os.environ.get("HIPCC", "/opt/rocm/bin/hipcc"), *HIPCC_FLAGS]
    with tempfile.TemporaryDirectory() as tmp:
        objects = [os.path.join(tmp, os.path.basename(src) + ".o") for src in sources]
        compiles = [[*hipcc, "-I", os.path.join(ROOT, "include"), "-c", "-o", obj, src]
                    for src, obj in zip(sources, objects)]
        with ThreadPoolExecutor(4) as pool:
            list(pool.map(lambda cmd: _run(cmd, verbose), compiles))
        _run([*hipcc, "-shared", "-o", out + ".tmp", *objects], verbose)
    os.replace(out + ".tmp", out)
    return out


def _host_module(source, out, verbose):
    """Compile a Python module of host code against torch's headers and libraries."""
    import sysconfig

    import torch
    home = os.path.dirname(torch.__file__)
    _run([os.environ.get("HIPCC", "/opt/rocm/bin/hipcc"), "-x", "c++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall",
          "-D__HIP_PLATFORM_AMD__=1", "-DUSE_ROCM=1", "-I", os.path.join(ROOT, "include"), "-I", os.path.join(home, "include"),
          "-I", "/opt/rocm/include", "-I", sysconfig.get_path("include"), "-o", out + ".tmp", source,
          "-L", os.path.join(home, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_hip"], verbose)
    os.replace(out + ".tmp", out)


def build(verbose: bool = False) -> str:
    """Compile libiq.so (the library), libiq_bench.so (the benchmark's
    reference copy kernel) and _fast.so (the binding's short calls)."""
    _hipcc(BENCH_SOURCES, BENCH_OUT, verbose)
    _host_module(FAST_SOURCE, FAST_OUT, verbose)
    return _hipcc(SOURCES, OUT, verbose)


if __name__ == "__main__":
    print(build(verbose=True))
