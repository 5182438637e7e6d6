"""Group norm takes the form that was measured to be faster (no GPU needed:
tests/host/block_plans.cpp asks the plans)."""
import os
import subprocess

import pytest

from test_sequence_launches import CSRC, HIPCC, ROOT, _run


def test_forms_at_measured_sizes(tmp_path):
    if not os.path.exists(HIPCC):
        pytest.skip("hipcc not available")
    exe = str(tmp_path / "block_plans")
    _run([HIPCC, "--offload-arch=gfx950", "-O1", "-std=c++17", "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
          "-I", os.path.join(ROOT, "include"), "-I", CSRC, "-x", "hip", os.path.join(ROOT, "tests", "host", "block_plans.cpp"), "-o", exe])
    env = dict(os.environ, HIP_VISIBLE_DEVICES="", ROCR_VISIBLE_DEVICES="")
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120, env=env)
    assert r.returncode == 0 and " 0 failure(s)" in r.stdout, r.stdout[-4000:] + r.stderr[-2000:]
