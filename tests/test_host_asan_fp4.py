"""The host code of the MXFP4 x MXFP4 layer, of tokens by expert and of the
experts' products (api_fp4.cpp: argument checks, choice of form, workspaces)
built for the CPU with AddressSanitizer and UndefinedBehaviorSanitizer and
driven through its C entry points (tests/asan/host_driver_fp4.cpp), with stubs
for the kernel launchers that write every byte their kernels write.  CPU only:
nothing touches a GPU."""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "mxfp8_block_scaled_amd", "csrc")


@pytest.mark.skipif(shutil.which("g++") is None or not os.path.isdir("/opt/rocm/include"),
                    reason="needs g++ and the ROCm headers")
def test_fp4_host_code_under_asan(tmp_path):
    exe = str(tmp_path / "host_driver_fp4")
    cmd = ["g++", "-std=c++17", "-O1", "-g", "-fno-omit-frame-pointer", "-fsanitize=address,undefined",
           "-fno-sanitize-recover=all", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
           "-I" + os.path.join(ROOT, "include"), "-I" + CSRC, os.path.join(CSRC, "api_fp4.cpp"),
           os.path.join(ROOT, "tests", "asan", "host_driver_fp4.cpp"), "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-4000:]
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:abort_on_error=0", UBSAN_OPTIONS="print_stacktrace=1")
    r = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=300)
    assert r.returncode == 0, (r.stdout[-2000:], r.stderr[-6000:])
    assert "host driver ok" in r.stdout
