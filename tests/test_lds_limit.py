"""The limit of a kernel's dynamic LDS is set on every device that launches it (CPU only: see
lds_limit_main.cpp), and by that function alone."""
import glob
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "bit_block_quant_amd", "csrc")


@pytest.mark.skipif(shutil.which("g++") is None or not os.path.isdir("/opt/rocm/include"),
                    reason="g++ or the HIP headers not available")
def test_set_on_each_device(tmp_path):
    exe = str(tmp_path / "lds_limit")
    build = subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Wextra", "-Werror", "-D__HIP_PLATFORM_AMD__", "-isystem", "/opt/rocm/include",
                            os.path.join(ROOT, "tests", "lds_limit_main.cpp"), "-o", exe], capture_output=True, text=True)
    assert build.returncode == 0, build.stderr
    run = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert run.returncode == 0 and "clean" in run.stdout, run.stdout + run.stderr


def test_set_nowhere_else():
    found = [os.path.basename(f) for f in glob.glob(os.path.join(CSRC, "*")) if "hipFuncSetAttribute" in open(f).read()]
    assert found == ["qblk_lds.h"]
