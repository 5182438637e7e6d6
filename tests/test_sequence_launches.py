"""Every launch of attention and its gradients stays within the runtime's
limit of threads up to the documented sizes, and layer norm's gradients ask
for the workspace of the workgroups that they launch (no GPU needed: the
kernels' regular build linked with tests/host/launch_checks.cpp, whose own
launch call only records the grid)."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "deformable_convolution_amd", "csrc")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")


def _run(cmd):
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, "%s\n%s%s" % (" ".join(cmd), r.stdout[-3000:], r.stderr[-3000:])


def test_launches_within_the_documented_limits(tmp_path):
    if not os.path.exists(HIPCC):
        pytest.skip("hipcc not available")
    kernels = [os.path.join(CSRC, "_build", f) for f in ("k_attention.o", "k_attention_bwd.o", "k_layernorm.o")]
    if not all(os.path.exists(o) for o in kernels):
        from deformable_convolution_amd.csrc import build
        build.build()
    obj, exe = str(tmp_path / "launch_checks.o"), str(tmp_path / "launch_checks")
    _run([HIPCC, "--offload-arch=gfx950", "-O1", "-std=c++17", "-fPIC", "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
          "-I", os.path.join(ROOT, "include"), "-I", CSRC, "-x", "hip", "-c", os.path.join(ROOT, "tests", "host", "launch_checks.cpp"),
          "-o", obj])
    _run([HIPCC, "--offload-arch=gfx950", obj, *kernels, "-o", exe])
    env = dict(os.environ, HIP_VISIBLE_DEVICES="", ROCR_VISIBLE_DEVICES="")
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120, env=env)
    assert r.returncode == 0 and " 0 failure(s)" in r.stdout, r.stdout[-4000:] + r.stderr[-2000:]
