"""The workspaces and addresses of group norm and the gated recurrence (no GPU
needed: the kernels' regular build linked with tests/host/block_memory.cpp, which
includes the recurrence's address arithmetic)."""
import os
import subprocess

import pytest

from test_sequence_launches import CSRC, HIPCC, ROOT, _run


def test_workspaces_and_rows(tmp_path):
    if not os.path.exists(HIPCC):
        pytest.skip("hipcc not available")
    kernels = [os.path.join(CSRC, "_build", f) for f in ("k_groupnorm.o", "k_groupnorm_bwd.o")]
    if not all(os.path.exists(o) for o in kernels):
        from deformable_convolution_amd.csrc import build
        build.build()
    obj, exe = str(tmp_path / "block_memory.o"), str(tmp_path / "block_memory")
    _run([HIPCC, "--offload-arch=gfx950", "-O1", "-std=c++17", "-fPIC", "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops", "-w",
          "-I", os.path.join(ROOT, "include"), "-I", CSRC, "-x", "hip", "-c", os.path.join(ROOT, "tests", "host", "block_memory.cpp"),
          "-o", obj])
    _run([HIPCC, "--offload-arch=gfx950", obj, *kernels, "-o", exe])
    env = dict(os.environ, HIP_VISIBLE_DEVICES="", ROCR_VISIBLE_DEVICES="")
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120, env=env)
    assert r.returncode == 0 and " 0 failure(s)" in r.stdout, r.stdout[-4000:] + r.stderr[-2000:]
