"""How exact the sums of the microscaled products are, and scales near both ends of their range.

In units of u = 2^-24 of sum|w x|, per result:

MXFP4 activations: a block's products are multiples of 1/4 of its scale, at most 36 each and
32 of them, so its sum is exact; adding up nb blocks and then at most min(nb, 16) waves' or
splits' parts takes as many roundings: nb + min(nb, 16).  With one scale everywhere all partial
sums are multiples of 1/4 below 2^22 of it, and the result is exact.

MXFP8 activations with fp32 results: k products (exact in fp32: 2 by 4 bits) and as many
additions: k.  Their elements are bf16 numbers on the way, multiples of 2^-133: an e4m3
element under one of the lowest scales may move by 2^-133, 2^-133 * sum|w| in a result.

16-bit results: test_gpu_mx_forms.py's bounds.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from test_gpu_mx import TYPES, q  # noqa: E402, F401
from test_gpu_mx_forms import check, wide  # noqa: E402

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def operand(rng, name, rows, k, low, high):
    """Random codes (no NaN) under scale bytes from low to high."""
    code = np.arange(256) if name == "mxfp4" else np.array([b for b in range(256) if b & 127 != 127])
    c = torch.from_numpy(rng.choice(code, (rows, k // 2 if name == "mxfp4" else k)).astype(np.uint8)).cuda()
    s = torch.from_numpy(rng.integers(low, high + 1, (rows, k // 32)).astype(np.uint8)).cuda()
    return (c if name == "mxfp4" else c.view(torch.float8_e4m3fn)), s


def check_sums(y, W, X, name):
    k = W.shape[1]
    ref, mag = X @ W.T, X.abs() @ W.abs().T
    bound = (k if name == "mxfp8" else k // 32 + min(k // 32, 16)) * U * mag + 2.0 ** -149
    if name == "mxfp8":
        bound = bound + 2.0 ** -133 * W.abs().sum(1)
    err = (y.double() - ref).abs()
    assert torch.all(err <= bound), ((err / mag).max() / U).item()


@pytest.mark.parametrize("span", [0, 8, 24, 60])
@pytest.mark.parametrize("n", [4, 20, 70, 130])
@pytest.mark.parametrize("k", [32, 64, 128, 256, 1024, 4096])
@pytest.mark.parametrize("name", ["mxfp4", "mxfp8"])
def test_sums_as_fp32_adds(q, name, k, n, span):  # noqa: F811
    """Blocks' scales up to 2^span apart in either operand."""
    rng = np.random.default_rng(k + n + span)
    m, low, high = 300, 127 - span // 2, 127 + span // 2
    wq, ws = operand(rng, "mxfp4", m, k, low, high)
    xq, xs = operand(rng, name, n, k, low, high)
    y, W, X = q.gemm_mxfp4(wq, ws, xq, xs), wide(wq, ws), wide(xq, xs)
    if span == 0 and name == "mxfp4":
        assert torch.equal(y.double(), X @ W.T)
    check_sums(y, W, X, name)


# the lowest and highest bytes that the quantizers make: 0, 252 (e2m1), 246 (e4m3)
ENDS = [(0, 0, 200, 200), (200, 200, 0, 0), (0, 8, 190, 230), (190, 230, 0, 8), (60, 70, 60, 70), (240, 252, 90, 100), (90, 100, 238, 246)]


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("n", [3, 20, 70])
@pytest.mark.parametrize("ends", ENDS)
@pytest.mark.parametrize("name", ["mxfp4", "mxfp8"])
def test_scales_at_the_ends(q, name, ends, n, out):  # noqa: F811
    rng = np.random.default_rng(sum(ends) + n)
    wq, ws = operand(rng, "mxfp4", 300, 256, *ends[:2])
    xq, xs = operand(rng, name, n, 256, *ends[2:])
    y, W, X = q.gemm_mxfp4(wq, ws, xq, xs, dtype=TYPES[out]), wide(wq, ws), wide(xq, xs)
    assert torch.isfinite(y).all()
    if out == "f32":
        check_sums(y, W, X, name)
    else:
        check(y, W, X, name)
