"""Build the gfx950 shared library libecho_amd.so in-tree with hipcc.

Flags that matter for the results:
  -ffp-contract=off        no a*b+c is fused except the dequantizer's explicit fmaf
  -fhip-fp32-correctly-rounded-divide-sqrt
                           IEEE division (the quantizer step and its reciprocal)
  -target-feature -packed-fp32-ops
                           no packed fp32 instructions are generated
fp32 denormals are kept (no -fgpu-flush-denormals-to-zero).
"""
from __future__ import annotations

import os
import subprocess
import tempfile
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
SOURCES = [os.path.join(CSRC, f) for f in ("echo_api.hip", "echo_kernels.hip", "echo_kv_api.hip",
                                           "echo_kv_cache.hip", "echo_kv_plan.hip", "echo_kv_attention.hip")]
HEADERS = [os.path.join(ROOT, "include", "echo.h")] + [
    os.path.join(CSRC, f) for f in ("echo_internal.h", "echo_kv_internal.h", "echo_kv_device.h")]
# The attention kernel is compiled once for every code width and head size.
FORMS = {"echo_kv_attention.hip": [[f"-DECHO_KV_BITS={bits}", f"-DECHO_KV_HEAD_DIM={dim}"]
                                   for bits in (4, 8) for dim in (256, 128, 64)]}
ARCH = "gfx950"


def library_path() -> str:
    return os.path.join(HERE, "libecho_amd.so")


def hipcc_flags() -> list[str]:
    return ["--offload-arch=" + ARCH, "-O3", "-std=c++17", "-fPIC", "-shared",
            "-ffp-contract=off", "-fhip-fp32-correctly-rounded-divide-sqrt",
            "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
            "-Wall", "-I", os.path.join(ROOT, "include"), "-I", CSRC]


def build(verbose: bool = False) -> str:
    """Compile every source to an object, several at a time, and link them."""
    out = library_path()
    hipcc, flags = "/opt/rocm/bin/hipcc", hipcc_flags()
    compile_flags = [f for f in flags if f != "-shared"] + ["-c"]
    units = [(src, form) for src in reversed(SOURCES) for form in FORMS.get(os.path.basename(src), [[]])]

    def run(cmd):
        if verbose:
            print(" ".join(cmd), flush=True)
        subprocess.run(cmd, check=True)

    with tempfile.TemporaryDirectory() as tmp:
        objects = [os.path.join(tmp, f"{i}.o") for i in range(len(units))]
        with ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as pool:
            list(pool.map(run, ([hipcc] + compile_flags + form + [src, "-o", obj]
                                for (src, form), obj in zip(units, objects))))
        run([hipcc, "--offload-arch=" + ARCH, "-shared", "-fPIC"] + objects + ["-o", out + ".tmp"])
    os.replace(out + ".tmp", out)
    return out


if __name__ == "__main__":
    print(build(verbose=True))
