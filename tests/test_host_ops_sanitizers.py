"""The host code of the operators' entry points (tsc_verify.h, tsc_train.h) under AddressSanitizer
and UndefinedBehaviorSanitizer (no GPU): compiled with both on the host pass only, the kernels as
usual and never launched; tests/host_ops_check.c calls every entry point with invalid and boundary
arguments. Any sanitizer report fails the test."""
import os
import subprocess

import pytest

from tests.test_host_sanitizers import LLVM, ROOT, _tool


def test_host_entry_points_under_asan_and_ubsan(tmp_path):
    hipcc, clang = _tool("hipcc"), os.path.join(LLVM, "clang")
    if not os.path.exists(clang):
        pytest.skip("the ROCm clang is needed for the sanitizer runtimes")
    package = os.path.join(ROOT, "top_support_capture_amd")
    inc = ["-I", os.path.join(ROOT, "include"), "-I", os.path.join(package, "csrc"),
           "-I", os.path.join(package, "csrc_ops")]
    lib = tmp_path / "libops_hostsan.so"
    san = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
           "-Xarch_host", "-fno-sanitize-recover=undefined", "-Xarch_host", "-fno-omit-frame-pointer"]
    subprocess.run([hipcc, "--offload-arch=gfx950", "-std=c++17", "-O1", "-g",
                    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
                    "-fPIC", "-shared", *san, *inc, "-o", str(lib),
                    os.path.join(package, "csrc_ops", "ops_api.hip")],
                   check=True, capture_output=True, timeout=600)
    exe = tmp_path / "host_ops_check"
    subprocess.run([clang, "-fsanitize=address,undefined", "-fno-sanitize-recover=undefined", "-g",
                    "-O1", *inc, os.path.join(ROOT, "tests", "host_ops_check.c"), str(lib),
                    f"-Wl,-rpath,{tmp_path}", "-o", str(exe)],
                   check=True, capture_output=True, timeout=300)
    env = dict(os.environ,
               ASAN_OPTIONS="detect_leaks=0:abort_on_error=0:exitcode=99",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1:exitcode=98")
    r = subprocess.run([str(exe)], env=env, capture_output=True, text=True, timeout=300)
    out = r.stdout + r.stderr
    assert "AddressSanitizer" not in out and "runtime error" not in out, out[-4000:]
    assert r.returncode == 0, out[-4000:]
    assert "host operator checks: 0 failure(s)" in r.stdout
