"""No kernel of the feed-forward operators keeps registers in memory (CPU only:
the sources are compiled for gfx950 and the compiler's report is read).

Their loops count the loads that are under way, and wait for the oldest; a
register read back from memory waits for all of them.
"""
import importlib.util
import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
_spec = importlib.util.spec_from_file_location("qblk_build", os.path.join(ROOT, "bit_block_quant_amd", "build.py"))
build = importlib.util.module_from_spec(_spec)  # without the package, which needs the built library
_spec.loader.exec_module(build)
HIPCC = build.hipcc()


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc not available")
@pytest.mark.parametrize("source,kernels", [("qblk_moe.hip", ("k_moe_up", "k_moe_down")), ("qblk_f8.hip", ("k_f8_few", "k_f8_tile"))])
def test_no_spills(source, kernels, tmp_path):
    cmd = [HIPCC, *build.FLAGS, "--cuda-device-only", "-c", os.path.join(build.CSRC, source), "-o", str(tmp_path / "o"),
           "-Rpass-analysis=kernel-resource-usage"]
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr
    found = re.findall(r"Function Name: (\S+).*?ScratchSize \[bytes/lane\]: (\d+).*?VGPRs Spill: (\d+)", r.stderr, re.S)
    for k in kernels:
        assert any(k in name for name, _, _ in found), k
    assert not [f for f in found if f[1:] != ("0", "0")]
