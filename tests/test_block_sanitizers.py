"""The host code of group norm and the gated recurrence (api_block.hip:
validation, planning, the C ABI) under AddressSanitizer and
UndefinedBehaviorSanitizer, as test_sequence_sanitizers.py does for the other
sequence operators' (no GPU needed): compiled with both on its host side,
linked with the regular build's kernels, and driven by
tests/host/block_checks.cpp with sizes, strides and arguments at the integers'
limits.  Any sanitizer report fails the run."""
import os
import subprocess

import pytest

from test_sequence_sanitizers import CLANG, CSRC, HIPCC, ROOT, SAN_HOST, _run


def test_host_validation_is_sanitizer_clean(tmp_path):
    if not (os.path.exists(HIPCC) and os.path.exists(CLANG)):
        pytest.skip("hipcc / clang not available")
    d = str(tmp_path)
    kernels = [os.path.join(CSRC, "_build", f) for f in ("k_groupnorm.o", "k_groupnorm_bwd.o", "k_recurrence.o")]
    if not all(os.path.exists(o) for o in kernels):
        from deformable_convolution_amd.csrc import build
        build.build()
    api = os.path.join(d, "api_block_san.o")
    _run([HIPCC, "--offload-arch=gfx950", "-O1", "-g", "-std=c++17", "-fPIC", "-Xclang", "-target-feature", "-Xclang",
          "-packed-fp32-ops", *SAN_HOST, "-I", os.path.join(ROOT, "include"), "-c", os.path.join(CSRC, "api_block.hip"), "-o", api])
    _run([CLANG, "-shared", "-fPIC", "-fsanitize=address,undefined", "-shared-libsan", "-o", os.path.join(d, "libblock_san.so"), api,
          *kernels, "-L/opt/rocm/lib", "-lamdhip64", "-Wl,-rpath,/opt/rocm/lib"])
    rt = os.path.dirname(subprocess.run(["/opt/rocm/llvm/bin/clang", "-print-file-name=libclang_rt.asan-x86_64.so"],
                                        capture_output=True, text=True).stdout.strip())
    exe = os.path.join(d, "block_checks")
    _run([CLANG, "-O1", "-g", "-std=c++17", "-fsanitize=address,undefined", "-fno-sanitize-recover=undefined", "-shared-libsan", "-I",
          os.path.join(ROOT, "include"), os.path.join(ROOT, "tests", "host", "block_checks.cpp"), "-o", exe, "-L", d, "-lblock_san",
          "-Wl,-rpath," + d, "-Wl,-rpath," + rt])
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=0", UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1",
               HIP_VISIBLE_DEVICES="", ROCR_VISIBLE_DEVICES="")
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300, env=env)
    out = r.stdout + r.stderr
    assert "ERROR: AddressSanitizer" not in out and "runtime error" not in out, out[-4000:]
    assert r.returncode == 0 and " 0 failure(s)" in out, out[-4000:]
