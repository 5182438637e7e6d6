"""Build libdc1d.so (gfx950) in-tree with hipcc.

    python -m deformable_convolution_amd.csrc.build        # or build() from Python

Every source is compiled for gfx950 only, with packed-fp32 instruction
selection disabled (scalar fp32 arithmetic only), and linked into
``deformable_convolution_amd/libdc1d.so``.  The sequence operators' Python
binding (host code only) becomes ``deformable_convolution_amd/_seq.so``.
"""
from __future__ import annotations

import os
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
PKG = os.path.dirname(HERE)
ROOT = os.path.dirname(PKG)
OUT = os.path.join(PKG, "libdc1d.so")
SOURCES = ["api.hip", "k_direct.hip", "k_backward.hip", "k_packed.hip", "k_dc2d.hip", "k_mfma.hip", "k_mfma_f32.hip", "k_mfma_f32_mask.hip", "k_mfma_bf16.hip",
           "k_mfma_bf16_mask.hip", "k_mfma_wide.hip", "k_heads.hip", "api_seq.hip", "k_layernorm.hip",
           "k_rotary.hip", "k_attention.hip", "k_attention_bwd.hip", "api_block.hip", "k_groupnorm.hip", "k_groupnorm_bwd.hip",
           "k_recurrence.hip"]
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-result", "-I", os.path.join(ROOT, "include"),
]


BIND = os.path.join(PKG, "_seq.so")


def build_binding(verbose: bool = False) -> str:
    """_seq.so: bind_seq.cpp against this interpreter and torch."""
    import torch
    from torch.utils import cpp_extension
    tmp = BIND + ".tmp%d" % os.getpid()
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", "-I", os.path.join(ROOT, "include"),
           "-I", sysconfig.get_paths()["include"]]
    for d in cpp_extension.include_paths():
        cmd += ["-isystem", d]
    cmd += [os.path.join(HERE, "bind_seq.cpp"), "-o", tmp, "-L", os.path.join(os.path.dirname(torch.__file__), "lib"),
            "-lc10", "-ltorch_cpu", "-ltorch_python"]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("g++ failed for bind_seq.cpp:\n%s" % r.stderr)
    os.replace(tmp, BIND)
    return BIND


def build(verbose: bool = False) -> str:
    objdir = os.path.join(HERE, "_build")
    os.makedirs(objdir, exist_ok=True)

    def compile_one(src):
        obj = os.path.join(objdir, src.replace(".hip", ".o"))
        cmd = [HIPCC, *FLAGS, "-c", os.path.join(HERE, src), "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("hipcc failed for %s:\n%s" % (src, r.stderr))
        return obj

    with ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        binding = ex.submit(build_binding, verbose)
        objs = list(ex.map(compile_one, SOURCES))
        binding.result()
    tmp = OUT + ".tmp%d" % os.getpid()
    cmd = [HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n%s" % r.stderr)
    os.replace(tmp, OUT)
    return OUT


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
