"""The host code of the 128-block FP8 layer, the weight gradient and the
balance loss (api_b128.cpp: argument checks, choice of form, workspace and kept
buffers) built for the CPU with AddressSanitizer and
UndefinedBehaviorSanitizer and driven through its C entry points
(tests/asan/host_driver_b128.cpp), with stubs for the kernel launchers that
write every byte their kernels write.  CPU only: nothing touches a GPU."""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "mxfp8_block_scaled_amd", "csrc")


@pytest.mark.skipif(shutil.which("g++") is None or not os.path.isdir("/opt/rocm/include"),
                    reason="needs g++ and the ROCm headers")
def test_b128_host_code_under_asan(tmp_path):
    exe = str(tmp_path / "host_driver_b128")
    cmd = ["g++", "-std=c++17", "-O1", "-g", "-fno-omit-frame-pointer", "-fsanitize=address,undefined",
           "-fno-sanitize-recover=all", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
           "-I" + os.path.join(ROOT, "include"), "-I" + CSRC, os.path.join(CSRC, "api_b128.cpp"),
           os.path.join(ROOT, "tests", "asan", "host_driver_b128.cpp"), "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-4000:]
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:abort_on_error=0", UBSAN_OPTIONS="print_stacktrace=1")
    r = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=300)
    assert r.returncode == 0, (r.stdout[-2000:], r.stderr[-6000:])
    assert "host driver ok" in r.stdout
