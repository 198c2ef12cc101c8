"""The forms of the microscaled products that test_gpu_mx_forms.py's sizes do not reach, and
which forms the sizes of both files run: a form that no size runs any more fails here.

The choice is an estimate's for 256 compute units; it is read from what the library logs of its
launches (QBLK_LOG=1, read once a process: hence a process of its own).
"""
import json
import os
import re
import subprocess
import sys

import pytest

torch = pytest.importorskip("torch")

from test_gpu_mx import TYPES, act, q  # noqa: E402, F401
from test_gpu_mx_forms import EXACT, FEW, TILES4, TILES8, TILES16, check, operands, run, wide  # noqa: E402

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# (m, k, n), and the form that the size is there for
WIDE8 = [(38460, 7712, 11), (661, 8416, 5377),  # 256 x 64
         (33510, 5568, 5), (6549, 23520, 169),  # split
         (3499, 8704, 5399), (28714, 7808, 540)]  # the rest of a cut
EXACT_SPLIT = [(5510, 3104, 69), (33385, 6112, 18), (131, 3200, 2719)]  # 256 x 128, split: one round, two; tokens past the last
MIXED = [(300, 4096, 1), (4100, 2080, 3), (300, 2080, 6)]  # 16 waves and 8, quantized in the product's launch

FORMS = {f"f4 {s}{p}" for p in ("", " split") for s in ("256x256 stages=2", "256x64 stages=3", "128x128 stages=2", "128x128 stages=3",
                                                        "128x64 stages=2", "128x64 stages=3", "64x64 stages=3")}
FORMS |= {f"f8 {s}{p}" for p in ("", " split") for s in ("256x256 stages=3", "256x128 stages=4", "256x64 stages=5", "128x128 stages=3",
                                                         "128x64 stages=4", "64x64 stages=5")}
FORMS |= {f"exact {s} stages=4{p}" for p in ("", " split") for s in ("256x128", "128x64")}
FORMS |= {f"few {kind} T=1 waves={waves} x={x}" for kind in ("f4", "f8", "f8 exact") for waves in (8, 16) for x in range(4)}
FORMS |= {f"few f4 T=2 waves={waves} x=3" for waves in (8, 16)}

CHILD = """
import json, sys
sys.path.insert(0, sys.argv[1])
import torch
import bit_block_quant_amd as q
types = [torch.float32, torch.float16, torch.bfloat16]
for m, k, n, f8, x, y in json.load(sys.stdin):
    w, ws = torch.zeros(m, k // 2, dtype=torch.uint8, device="cuda"), torch.zeros(m, k // 32, dtype=torch.uint8, device="cuda")
    if x < 3:
        q.linear_mxfp4(torch.zeros(n, k, dtype=types[x], device="cuda"), w, ws, act=q.ACT_MXFP8 if f8 else q.ACT_MXFP4, dtype=types[y])
    else:
        c = torch.zeros(n, k if f8 else k // 2, dtype=torch.uint8, device="cuda")
        q.gemm_mxfp4(w, ws, c.view(torch.float8_e4m3fn) if f8 else c, torch.zeros(n, k // 32, dtype=torch.uint8, device="cuda"), dtype=types[y])
torch.cuda.synchronize()
"""


def test_every_form_is_run(q):  # noqa: F811
    calls = [(*s, 0, 3, (s[0] + s[2]) % 3) for s in TILES4] + [(*s, 1, 3, 1 + (s[0] + s[2]) % 2) for s in TILES8 + WIDE8]
    calls += [(*s, 1, 3, 0) for s in EXACT + EXACT_SPLIT] + [(*s, f8, 3, y) for s in TILES16 + FEW for f8 in (0, 1) for y in (0, 2)]
    calls += [(*s, f8, x, y) for s in MIXED for f8 in (0, 1) for x in range(3) for y in range(3)]
    r = subprocess.run([sys.executable, "-c", CHILD, ROOT], input=json.dumps(calls), capture_output=True, text=True, timeout=100,
                       env={**os.environ, "QBLK_LOG": "1"})
    assert r.returncode == 0, r.stderr[-2000:]
    tiles = re.findall(r"qblk: mx tile (\S+ \S+ stages=\d+(?: split)?) m=", r.stderr)
    few = [f"few {f}{e} T={t} waves={v} x={x}" for f, t, v, x, e in
           re.findall(r"qblk: mx few (f\d) m=\d+ k=\d+ n=\d+ T=(\d) waves=(\d+) rows=\d+ x=(\d)( exact)? lds=", r.stderr)]
    assert set(tiles) | set(few) == FORMS, (FORMS - set(tiles) - set(few), (set(tiles) | set(few)) - FORMS)
    wide8 = re.findall(r"mx tile f8 256x64 stages=5( split)? m=(\d+) k=(\d+) n=(\d+)", r.stderr)
    assert {tuple(map(int, s[1:])) for s in wide8} == set(WIDE8)
    split = re.findall(r"mx tile exact 256x128 stages=4 split m=(\d+) k=(\d+) n=(\d+)", r.stderr)
    assert {tuple(map(int, s)) for s in split} == set(EXACT_SPLIT)


@pytest.mark.parametrize("m,k,n", WIDE8)
def test_wide_tiles_of_8_bits(q, m, k, n):  # noqa: F811
    run(q, m, k, n, "mxfp8", ["f16", "bf16"][(m + n) % 2])


@pytest.mark.parametrize("m,k,n", EXACT_SPLIT)
def test_split_tiles_with_exact_sums(q, m, k, n):  # noqa: F811
    run(q, m, k, n, "mxfp8", "f32")


@pytest.mark.parametrize("name", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("x_type", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("m,k,n", MIXED + [(300, 2080, 40)])
def test_results_of_another_type_than_x(q, m, k, n, x_type, name):  # noqa: F811
    wq, ws, _, _, x = operands(q, m, k, n, name)
    x = x.to(TYPES[x_type])
    X = wide(*getattr(q, f"quantize_{name}")(x))
    for dtype in ("f32", "f16", "bf16"):
        y = q.linear_mxfp4(x, wq, ws, act=act(q, name), dtype=TYPES[dtype])
        assert y.dtype == TYPES[dtype]
        check(y, wide(wq, ws), X, name)
