"""The sequence operators' host code (api_seq.hip: validation, planning, the C
ABI) under AddressSanitizer and UndefinedBehaviorSanitizer, as
test_host_sanitizers.py does for the convolutions' (no GPU needed): compiled
with both on its host side, linked with the regular build's kernels, and
driven by tests/host/sequence_checks.cpp with sizes, strides and arguments at
the integers' limits.  Any sanitizer report fails the run."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "deformable_convolution_amd", "csrc")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
CLANG = "/opt/rocm/llvm/bin/clang++"
SAN_HOST = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined", "-Xarch_host",
            "-fno-sanitize-recover=undefined", "-Xarch_host", "-fno-omit-frame-pointer"]


def _run(cmd):
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, "%s\n%s%s" % (" ".join(cmd), r.stdout[-3000:], r.stderr[-3000:])


def test_host_validation_is_sanitizer_clean(tmp_path):
    if not (os.path.exists(HIPCC) and os.path.exists(CLANG)):
        pytest.skip("hipcc / clang not available")
    d = str(tmp_path)
    kernels = [os.path.join(CSRC, "_build", f) for f in ("k_layernorm.o", "k_rotary.o", "k_attention.o", "k_attention_bwd.o")]
    if not all(os.path.exists(o) for o in kernels):
        from deformable_convolution_amd.csrc import build
        build.build()
    api = os.path.join(d, "api_seq_san.o")
    _run([HIPCC, "--offload-arch=gfx950", "-O1", "-g", "-std=c++17", "-fPIC", "-Xclang", "-target-feature", "-Xclang",
          "-packed-fp32-ops", *SAN_HOST, "-I", os.path.join(ROOT, "include"), "-c", os.path.join(CSRC, "api_seq.hip"), "-o", api])
    _run([CLANG, "-shared", "-fPIC", "-fsanitize=address,undefined", "-shared-libsan", "-o", os.path.join(d, "libseq_san.so"), api,
          *kernels, "-L/opt/rocm/lib", "-lamdhip64", "-Wl,-rpath,/opt/rocm/lib"])
    rt = os.path.dirname(subprocess.run(["/opt/rocm/llvm/bin/clang", "-print-file-name=libclang_rt.asan-x86_64.so"],
                                        capture_output=True, text=True).stdout.strip())
    exe = os.path.join(d, "sequence_checks")
    _run([CLANG, "-O1", "-g", "-std=c++17", "-fsanitize=address,undefined", "-fno-sanitize-recover=undefined", "-shared-libsan", "-I",
          os.path.join(ROOT, "include"), os.path.join(ROOT, "tests", "host", "sequence_checks.cpp"), "-o", exe, "-L", d, "-lseq_san",
          "-Wl,-rpath," + d, "-Wl,-rpath," + rt])
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=0", UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1",
               HIP_VISIBLE_DEVICES="", ROCR_VISIBLE_DEVICES="")
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300, env=env)
    out = r.stdout + r.stderr
    assert "ERROR: AddressSanitizer" not in out and "runtime error" not in out, out[-4000:]
    assert r.returncode == 0 and " 0 failure(s)" in out, out[-4000:]
