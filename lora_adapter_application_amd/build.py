"""Compile the gfx950 HIP library ``liblora_mi355x.so`` in-tree.

    python -m lora_adapter_application_amd.build

The library is the C ABI of ``include/lora_mi355x.h``: the runtime
(``csrc/lora_runtime.cpp``), the low-rank kernels (``csrc/lora_kernels.hip``),
the saved-module kernels (``csrc/lora_saved.hip``), and the frozen part of a
layer: its host side (``csrc/lora_layer.cpp``), the 4-bit base products
(``csrc/lora_base.hip``) and rotary positions (``csrc/lora_rotary.hip``).
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
INCLUDE = os.path.join(ROOT, "include")
LIB_NAME = "liblora_mi355x.so"
LIB_PATH = os.path.join(PKG, LIB_NAME)
ARCH = "gfx950"

SOURCES = [os.path.join(CSRC, name) for name in
           ("lora_kernels.hip", "lora_saved.hip", "lora_base.hip", "lora_rotary.hip",
            "lora_runtime.cpp", "lora_layer.cpp")]

# Packed-fp32 instructions stay disabled for device code (the host pass warns
# that it does not know the feature; that is harmless).
HIPCC_FLAGS = ["--offload-arch=" + ARCH, "-O3", "-std=c++17", "-fPIC",
               "-Wall", "-Wno-unused-result",
               "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
               "-I", INCLUDE]


def hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", "hipcc"):
        if cand and (os.path.sep not in cand or os.path.exists(cand)):
            return cand
    raise RuntimeError("hipcc not found")


def build(verbose: bool = False) -> str:
    """Always recompile; returns the path of the shared library."""
    tmp = LIB_PATH + ".tmp"

    def run(cmd):
        if verbose:
            print(" ".join(cmd), flush=True)
        res = subprocess.run(cmd, capture_output=True, text=True)
        noise = "is not a recognized feature for this target"
        msgs = [l for l in (res.stdout + res.stderr).splitlines() if noise not in l]
        if res.returncode != 0:
            raise RuntimeError("hipcc failed:\n" + "\n".join(msgs))
        if verbose and msgs:
            print("\n".join(msgs))

    with tempfile.TemporaryDirectory() as objs:
        out = [os.path.join(objs, os.path.basename(s) + ".o") for s in SOURCES]
        with ThreadPoolExecutor(4) as pool:     # the sources beside each other
            list(pool.map(run, [[hipcc(), *HIPCC_FLAGS, "-c", "-o", o, s] for o, s in zip(out, SOURCES)]))
        run([hipcc(), "--offload-arch=" + ARCH, "-shared", "-o", tmp, *out])
    os.replace(tmp, LIB_PATH)
    return LIB_PATH


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
