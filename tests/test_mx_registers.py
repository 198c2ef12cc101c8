"""No kernel of the microscaled products and the norm keeps registers in memory (CPU
only: the sources are compiled for gfx950 and the compiler's report is read).

Their loops count the loads that are under way; a register read back from memory would
wait for all of them."""
import os
import re
import subprocess

import pytest

from test_ffn_registers import HIPCC, build


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc not available")
@pytest.mark.parametrize("source,kernel", [("qblk_mx.hip", "k_mx_few"), ("qblk_mx_tile.hip", "k_mx_tile"), ("qblk_norm.hip", "k_rmsnorm")])
def test_no_spills(source, kernel, tmp_path):
    cmd = [HIPCC, *build.FLAGS, "--cuda-device-only", "-c", os.path.join(build.CSRC, source), "-o", str(tmp_path / "o"),
           "-Rpass-analysis=kernel-resource-usage"]
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr
    found = re.findall(r"Function Name: (\S+).*?ScratchSize \[bytes/lane\]: (\d+).*?VGPRs Spill: (\d+)", r.stderr, re.S)
    assert any(kernel in name for name, _, _ in found)
    assert not [f for f in found if f[1:] != ("0", "0")]
