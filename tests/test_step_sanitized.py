"""Host code of a fine-tuning step's operators built with g++ under AddressSanitizer and UndefinedBehaviorSanitizer,
linked with stand-ins for the kernel launchers that check every workspace region (tests/step_sanitize/main.cpp). No GPU
code runs."""
import os
import shutil
import subprocess
import tempfile

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")
CSRC = os.path.join(ROOT, "rank_gemm_lora_amd", "csrc")


@pytest.mark.skipif(shutil.which("g++") is None or not os.path.exists(os.path.join(ROCM, "include", "hip")),
                    reason="needs g++ and the ROCm headers")
def test_host_code_under_sanitizers():
    with tempfile.TemporaryDirectory(prefix="lora_asan_") as tmp:
        exe = os.path.join(tmp, "step_sanitized")
        cmd = ["g++", "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
               "-fno-omit-frame-pointer", "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(ROCM, "include"),
               "-I", os.path.join(ROOT, "include"), "-I", CSRC, os.path.join(CSRC, "step_api.cpp"),
               os.path.join(ROOT, "tests", "step_sanitize", "main.cpp"), "-o", exe]
        r = subprocess.run(cmd, capture_output=True, text=True)
        assert r.returncode == 0, r.stderr[-4000:]
        env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:abort_on_error=0", UBSAN_OPTIONS="print_stacktrace=1")
        r = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=300)
        assert r.returncode == 0, (r.stdout[-2000:] + r.stderr[-2000:])
        assert ", 0 failures" in r.stdout
