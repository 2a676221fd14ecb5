"""Compile the gfx950 HIP library (libnvfp4.so) in-tree with hipcc."""
from __future__ import annotations

import hashlib
import os
import re
import subprocess
import sys
import tempfile
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libnvfp4.so")
SOURCES = [os.path.join(CSRC, "nvfp4_api.cpp"), os.path.join(CSRC, "nvfp4_plan.cpp"),
           os.path.join(CSRC, "nvfp4_sequence.cpp"), os.path.join(CSRC, "nvfp4_kernels.hip"), os.path.join(CSRC, "nvfp4_grouped.hip"),
           os.path.join(CSRC, "nvfp4_quantize.hip"), os.path.join(CSRC, "nvfp4_probe.hip"),
           os.path.join(CSRC, "nvfp4_noalloc.hip"), os.path.join(CSRC, "nvfp4_mx_api.cpp"),
           os.path.join(CSRC, "nvfp4_mx_quantize.hip"), os.path.join(CSRC, "nvfp4_mx_gemm.hip"),
           os.path.join(CSRC, "nvfp4_moe.hip")]
# the operators around the products of a layer (include/nvfp4_layer.h)
LAYER_SOURCES = [os.path.join(CSRC, f) for f in ("nvfp4_layer_api.cpp", "nvfp4_mx_fused.hip",
                                                 "nvfp4_mx_fused_grouped.hip", "nvfp4_mx_gated.hip",
                                                 "nvfp4_mx_moe.hip", "nvfp4_mx_short.hip", "nvfp4_norm.hip",
                                                 "nvfp4_norm_bf16.hip", "nvfp4_norm_f32.hip",
                                                 "nvfp4_norm_grad_bf16.hip", "nvfp4_norm_grad_f32.hip")]
# what the kernels that a plan table times, and their launches, are built from
KERNEL_FILES = [os.path.join(CSRC, f) for f in ("nvfp4_kernels.hip", "nvfp4_grouped.hip",
                                                "nvfp4_quantize.hip", "nvfp4_internal.h",
                                                "nvfp4_device.h", "nvfp4_quant_device.h")]

HIPCC_FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC", "-shared",
    # keep the compiler from emitting packed-FP32 VALU instructions
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    # kernels with plain arguments get the leading ones preloaded into scalar
    # registers before their waves start (the decode-sized kernels: one
    # memory round trip less per call)
    "-mllvm", "-amdgpu-kernarg-preload-count=16",
    "-Wall", "-Wno-unused-command-line-argument",
]


def hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", "hipcc"):
        if cand and (os.path.isabs(cand) and os.path.exists(cand) or not os.path.isabs(cand)):
            return cand
    return "hipcc"


_COMMENT = re.compile(r"//[^\n]*|/\*.*?\*/", re.S)


def build_id() -> str:
    """Hash of the kernel sources and compiler flags, comments and blank lines
    left out: a tuned plan table records the id of the kernels it timed."""
    h = hashlib.sha256(" ".join(HIPCC_FLAGS).encode())
    for path in KERNEL_FILES:
        text = _COMMENT.sub("", open(path).read())
        lines = [l.rstrip() for l in text.splitlines() if l.strip()]
        h.update(os.path.basename(path).encode() + b"\0" + "\n".join(lines).encode() + b"\0")
    return h.hexdigest()[:16]


def _hipcc(args: list[str], verbose: bool) -> None:
    cmd = [hipcc(), *HIPCC_FLAGS, f"-DNVFP4_BUILD_ID=\"{build_id()}\"", "-I", INCLUDE, "-I", CSRC, *args]
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    noise = "is not a recognized feature for this target"
    err = "\n".join(l for l in res.stderr.splitlines() if noise not in l)
    if res.returncode != 0:
        raise RuntimeError(f"hipcc failed ({res.returncode}):\n{err}")
    if verbose and err.strip():
        print(err, file=sys.stderr)


def build(verbose: bool = False) -> str:
    """Compiles every source, up to eight side by side, and links the library."""
    tmp = LIB + f".tmp{os.getpid()}"
    with tempfile.TemporaryDirectory() as d:
        sources = SOURCES + LAYER_SOURCES
        objects = [os.path.join(d, os.path.basename(s) + ".o") for s in sources]
        with ThreadPoolExecutor(min(8, os.cpu_count() or 1)) as pool:
            list(pool.map(lambda so: _hipcc(["-c", "-o", so[1], so[0]], verbose), zip(sources, objects)))
        _hipcc(["-o", tmp, *objects], verbose)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
