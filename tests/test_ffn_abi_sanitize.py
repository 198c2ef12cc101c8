"""The feed-forward operators' argument checks under AddressSanitizer and
UndefinedBehaviorSanitizer (host code only, no GPU): see
ffn_abi_sanitize_main.cpp and test_abi_sanitize.py."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.skipif(shutil.which("g++") is None or not os.path.isdir("/opt/rocm/include"),
                    reason="g++ or the HIP headers not available")
def test_ffn_abi_checks_under_sanitizers(tmp_path):
    exe = str(tmp_path / "ffn_abi_sanitize")
    cmd = ["g++", "-x", "c++", "-std=c++17", "-O1", "-g", "-Wall", "-Wextra", "-Werror",
           "-Wno-unused-parameter", "-Wno-unused-function", "-D__HIP_PLATFORM_AMD__",
           "-isystem", "/opt/rocm/include",
           "-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-fno-omit-frame-pointer",
           os.path.join(ROOT, "tests", "ffn_abi_sanitize_main.cpp"), "-o", exe]
    build = subprocess.run(cmd, capture_output=True, text=True)
    if build.returncode != 0 and "sanitize" in build.stderr and "cannot find" in build.stderr:
        pytest.skip("sanitizer runtime not installed")
    assert build.returncode == 0, build.stderr
    run = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert run.returncode == 0, run.stdout + run.stderr
    assert "clean" in run.stdout
