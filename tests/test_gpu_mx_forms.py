"""The microscaled products' forms one by one, at sizes whose rows, tokens and columns
fill nothing evenly, with poisoned memory around every output; the quantizers' and the
norm's outputs likewise; and operands past 2^32 bytes.

Bounds as in test_gpu_mx.py, with the reference products formed in 64 bits on the GPU.
Which form a size runs is the estimate's choice on 256 compute units; the sizes below
were picked from its formula, and a wrong choice would only test another form twice.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from test_gpu_ffn import MARGIN, Padded  # noqa: E402
from test_gpu_mx import D, E2M1, E4M3, HALF_ULP, TINY, TYPES, act, q  # noqa: E402, F401

pytestmark = pytest.mark.gpu


def wide(codes, scale):
    """The values of codes (rows, k/2 or k) as float64 on the GPU."""
    b = codes.view(torch.uint8)
    if codes.dtype == torch.uint8:
        table = torch.tensor(np.concatenate([E2M1, -E2M1])).cuda()
        v = torch.empty(b.shape[0], 2 * b.shape[1], dtype=torch.float64, device="cuda")
        v[:, ::2], v[:, 1::2] = table[(b & 15).long()], table[(b >> 4).long()]
    else:
        table = torch.tensor(np.concatenate([E4M3, [np.nan], -E4M3, [np.nan]])).cuda()
        v = table[b.long()]
    return v * torch.exp2(scale.view(torch.uint8).double() - 127).repeat_interleave(32, 1)


def check(y, W, X, name):
    """Per result: |y - ref| within the sums' bound, and half a unit of the type."""
    drop = 7 * 2.0 ** -13 if name == "mxfp8" and y.dtype != torch.float32 else 0.0
    for r in range(0, W.shape[0], 4096):  # (float64 products of some thousand rows at a time)
        ref, mag = X @ W[r:r + 4096].T, X.abs() @ W[r:r + 4096].abs().T
        over = (y[:, r:r + 4096].double() - ref).abs() - ((2e-5 + drop) * mag + HALF_ULP[y.dtype] * (ref.abs() + 2e-5 * mag) + TINY[y.dtype])
        assert over.max() <= 0, (over / mag).max().item()


def operands(q, m, k, n, name):  # noqa: F811
    gen = torch.Generator("cuda").manual_seed(m + k + n)
    w = torch.randn(m, k, device="cuda", generator=gen) * torch.exp(-3 * torch.rand(m, 1, device="cuda", generator=gen))
    x = torch.randn(n, k, device="cuda", generator=gen)
    x[:, torch.randint(0, k, (3,), device="cuda", generator=gen)] *= 20
    return *q.quantize_mxfp4(w), *getattr(q, f"quantize_{name}")(x), x


def run(q, m, k, n, name, dtype, linear=False):  # noqa: F811
    wq, ws, xq, xs, x = operands(q, m, k, n, name)
    size = n * m * (4 if dtype == "f32" else 2)
    raw = torch.full((size + 2 * MARGIN,), 0xFF, dtype=torch.uint8, device="cuda")
    out = raw[MARGIN:MARGIN + size].view(TYPES[dtype]).view(n, m)
    kind = act(q, name)
    if linear:
        room = q.lib().qblk_linear_mxfp4_workspace(m, k, n, kind)
        x = x.to(TYPES[dtype])
        xq, xs = getattr(q, f"quantize_{name}")(x)
    else:
        room = q.lib().qblk_gemm_mxfp4_workspace(m, k, n, kind)
    work = Padded(torch.zeros(max(16, room), dtype=torch.uint8, device="cuda"))
    for _ in range(2):  # what the first call left in the workspace changes nothing
        y = (q.linear_mxfp4(x, wq, ws, act=kind, out=out, workspace=work.t) if linear
             else q.gemm_mxfp4(wq, ws, xq, xs, out=out, workspace=work.t))
        check(y, wide(wq, ws), wide(xq, xs), name)
        assert torch.all(raw[:MARGIN] == 0xFF) and torch.all(raw[MARGIN + size:] == 0xFF) and work.intact()
        first = y.clone()
        out.fill_(7.0)
        work.t.fill_(0xFF)
    y = q.linear_mxfp4(x, wq, ws, act=kind) if linear else q.gemm_mxfp4(wq, ws, xq, xs, dtype=TYPES[dtype])
    assert torch.equal(y, first)


# (m, k, n): rows x tokens of a tile, whole or K split (or rows cut in two launches)
TILES4 = [(11189, 288, 641), (10993, 14400, 135),  # 256 x 256, split
          (11040, 3200, 258), (10991, 11008, 33),  # 256 x 64, split
          (10881, 288, 130), (2315, 6400, 65), (11029, 288, 321), (10916, 14400, 65),  # 128 x 128, split; two workgroups a unit
          (8486, 3200, 65), (4381, 14400, 33), (11354, 288, 259), (5451, 11008, 33),  # 128 x 64, likewise
          (103, 288, 33), (100, 3200, 33), (258, 1152, 5474), (131, 4128, 1615),  # 64 x 64, split
          (11831, 288, 1540), (3477, 3200, 5400), (10571, 288, 1564), (6075, 288, 3217), (11992, 288, 1282)]  # cut
TILES8 = [(11189, 288, 641), (8270, 14400, 129), (11003, 1152, 325), (8277, 6400, 67), (11040, 3200, 258), (6438, 11008, 132),
          (10881, 288, 130), (2311, 3200, 65), (8416, 1152, 65), (517, 14400, 65), (103, 288, 33), (100, 3200, 33),
          (11678, 1152, 1685), (3477, 3200, 5400), (7330, 1152, 2327), (10016, 1152, 1552), (7175, 288, 2178), (1421, 4128, 5487),
          (9369, 3200, 784)]
EXACT = [(11029, 288, 321), (130, 3200, 2312), (103, 288, 33), (102, 1152, 33)]  # 256 x 128, split; 128 x 64, split
# few tokens whose codes leave no room, or of many rows
TILES16 = [(300, 14400, 12), (8200, 8224, 12), (25003, 288, 5), (12805, 1056, 16), (70001, 96, 1)]


@pytest.mark.parametrize("m,k,n", TILES4)
def test_tiles_of_4_bits(q, m, k, n):  # noqa: F811
    run(q, m, k, n, "mxfp4", ["f32", "f16", "bf16"][(m + n) % 3])


@pytest.mark.parametrize("m,k,n", TILES8)
def test_tiles_of_8_bits(q, m, k, n):  # noqa: F811
    run(q, m, k, n, "mxfp8", ["f16", "bf16"][(m + n) % 2])


@pytest.mark.parametrize("name", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("m,k,n", TILES16)
def test_tiles_of_few_tokens(q, m, k, n, name):  # noqa: F811
    for dtype in ("f32", "bf16"):
        run(q, m, k, n, name, dtype)
        if n > 4:
            run(q, m, k, n, name, dtype, linear=True)


@pytest.mark.parametrize("m,k,n", EXACT)
def test_tiles_with_exact_sums(q, m, k, n):  # noqa: F811
    run(q, m, k, n, "mxfp8", "f32")


@pytest.mark.parametrize("name", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("k", [32, 64, 96, 128, 160, 224, 256, 288, 480, 512, 544, 736, 1024, 1056])
def test_tiles_of_every_tail(q, k, name):  # noqa: F811
    """Columns that end inside a stage, a group of stages and a load of scales."""
    for dtype in ("f32", "bf16"):
        run(q, 140, k, 70, name, dtype)
        run(q, 140, k, 70, name, dtype, linear=True)


# (m, k, n): 16 waves or 8, one to three workgroups a compute unit, several turns of 16 rows, 32 tokens
FEW = [(300, 4096, 1), (4100, 2080, 3), (20003, 1056, 3), (700, 992, 16), (12345, 288, 9), (5003, 8192, 16), (700, 6144, 16),
       (2000, 1056, 28), (300, 2400, 25), (40001, 512, 2), (12805, 288, 4), (12005, 4096, 10), (700, 992, 20),
       (4000, 4096, 8), (300, 2080, 6)]


@pytest.mark.parametrize("name,dtype", [("mxfp4", "f32"), ("mxfp4", "f16"), ("mxfp8", "bf16"), ("mxfp8", "f32")])
@pytest.mark.parametrize("m,k,n", FEW)
def test_few_tokens(q, m, k, n, name, dtype):  # noqa: F811
    run(q, m, k, n, name, dtype)
    if n <= 8:
        run(q, m, k, n, name, dtype, linear=True)


@pytest.mark.parametrize("name", ["mxfp4", "mxfp8"])
def test_codes_of_all_kinds(q, name):  # noqa: F811
    """Every finite code in both operands, scales over many binades."""
    rng = np.random.default_rng(5)
    codes = np.arange(256) if name == "mxfp4" else np.array([b for b in range(256) if b & 127 != 127])
    for m, k, n in ((130, 512, 3), (257, 1152, 20), (300, 736, 90)):
        wq = torch.from_numpy(rng.integers(0, 256, (m, k // 2)).astype(np.uint8)).cuda()
        xq = torch.from_numpy(rng.choice(codes, (n, k // 2 if name == "mxfp4" else k)).astype(np.uint8)).cuda()
        xq = xq if name == "mxfp4" else xq.view(torch.float8_e4m3fn)
        ws, xs = (torch.from_numpy(rng.integers(100, 155, (r, k // 32)).astype(np.uint8)).cuda() for r in (m, n))
        for dtype in ("f32", "bf16"):
            check(q.gemm_mxfp4(wq, ws, xq, xs, dtype=TYPES[dtype]), wide(wq, ws), wide(xq, xs), name)


# ------------------------------------------------------- nothing beside the outputs
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("name", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("rows,k", [(1, 32), (3, 96), (257, 160), (1030, 1056)])
def test_quantizers_keep_to_their_outputs(q, rows, k, name, dtype):  # noqa: F811
    x = torch.randn(rows, k, device="cuda").to(TYPES[dtype])
    make = getattr(q, f"quantize_{name}")
    want, ws = make(x)
    out, scale = Padded(torch.zeros_like(want.view(torch.uint8))), Padded(torch.zeros_like(ws.view(torch.uint8)))
    make(x, out=out.t, scale=scale.t)
    assert torch.equal(out.t, want.view(torch.uint8)) and torch.equal(scale.t, ws.view(torch.uint8))
    values = Padded(torch.zeros_like(x))
    q.dequant_mx(want, ws, out=values.t)
    assert out.intact() and scale.intact() and values.intact()
    assert torch.equal(values.t, q.dequant_mx(want, ws, x.dtype))


@pytest.mark.parametrize("quant", ["f8", "i8", "mxfp8", "mxfp4"])
@pytest.mark.parametrize("n,h", [(1, 128), (5, 640), (3, 4224), (1100, 4224), (2, 9088), (1100, 6272), (300, 11264), (2, 40960)])
def test_norm_keeps_to_its_outputs(q, n, h, quant):  # noqa: F811
    """Every width's and number of rows' form, with all four outputs."""
    x, res = (torch.randn(n, h, device="cuda", dtype=torch.float16) for _ in range(2))
    w = torch.rand(h, device="cuda") + 0.5
    r = q.rmsnorm(x, w, res, quant=act(q, quant), y=True)
    t = (x.float() + res.float()).half()
    y = (t.double() / (t.double().square().mean(1, keepdim=True) + 1e-6).sqrt() * w.double())
    assert torch.equal(r.total, t)
    assert torch.all((r.y.double() - y).abs() <= (D + 2.0 ** -11) * y.abs() + 2.0 ** -24)
    outs = [Padded(torch.zeros_like(v.view(torch.uint8))) for v in (r.codes, r.scale, r.total, r.y)]
    got = q.rmsnorm(x, w, res, quant=act(q, quant), out=outs[0].t.view(r.codes.dtype), scale=outs[1].t.view(r.scale.dtype),
                    total=outs[2].t.view(x.dtype), y=outs[3].t.view(x.dtype))
    for a, b in zip(got, (r.codes, r.scale, r.total, r.y)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert all(o.intact() for o in outs)


@pytest.mark.parametrize("h", [8, 16, 24, 72])
def test_narrow_norms(q, h):  # noqa: F811
    for n in (1, 4, 9):
        x = torch.randn(n, h, device="cuda")
        w = torch.rand(h, device="cuda")
        y = q.rmsnorm(x, w, eps=1e-5, quant=None).y
        ref = x.double() / (x.double().square().mean(1, keepdim=True) + 1e-5).sqrt() * w.double()
        assert torch.all((y.double() - ref).abs() <= D * ref.abs())


def test_norm_without_columns(q):  # noqa: F811
    """As quantize_act_i8 of no columns: a scale of 0 for each row."""
    x, w = torch.empty(3, 0, device="cuda"), torch.empty(0, device="cuda")
    scale = torch.full((3,), 7.0, device="cuda")
    q.rmsnorm(x, w, quant=q.ACT_I8, scale=scale)
    assert torch.equal(scale, q.quantize_act_i8(x)[1]) and torch.equal(scale, torch.zeros(3, device="cuda"))
    for quant in (None, q.ACT_F8, q.ACT_MXFP8, q.ACT_MXFP4):
        r = q.rmsnorm(x, w, x, quant=quant, y=True)
        assert r.y.shape == (3, 0) and r.total.shape == (3, 0)


# ------------------------------------------------------------ past 2^32 bytes
def test_weights_past_32_bits(q):  # noqa: F811
    """4.3e9 bytes of codes: few tokens and many, rows at both ends and at 2^32 bytes."""
    m, k = (1 << 21) + 37, 4096
    gen = torch.Generator("cuda").manual_seed(1)
    wq = torch.randint(0, 256, (m, k // 2), dtype=torch.uint8, device="cuda", generator=gen)
    ws = torch.randint(118, 124, (m, k // 32), dtype=torch.uint8, device="cuda", generator=gen)
    rows = torch.tensor([0, 1, 15, 16, 4095, (1 << 21) - 1, 1 << 21, (1 << 21) + 1, m - 17, m - 1], device="cuda")
    for name, n, dtype in (("mxfp8", 1, "bf16"), ("mxfp4", 9, "f32"), ("mxfp4", 40, "bf16"), ("mxfp8", 130, "f16")):
        x = torch.randn(n, k, device="cuda")
        xq, xs = getattr(q, f"quantize_{name}")(x)
        y = q.gemm_mxfp4(wq, ws, xq, xs, dtype=TYPES[dtype])
        check(y[:, rows].contiguous(), wide(wq[rows], ws[rows]), wide(xq, xs), name)
        del y


def test_tokens_past_32_bits(q):  # noqa: F811
    """1.1 million tokens of 4096: the norm's 9 GB of values, codes past 2^32 bytes, and their product."""
    n, k, m = (1 << 20) + 1031, 4096, 72
    x = torch.randn(2048, k, device="cuda", dtype=torch.bfloat16).repeat(n // 2048 + 1, 1)[:n]
    x[-1] = 3.0
    w = torch.rand(k, device="cuda") + 0.5
    wq, ws = q.quantize_mxfp4(torch.randn(m, k, device="cuda"))
    at = torch.tensor([0, 1, 2047, 2048, (1 << 19) - 1, 1 << 19, (1 << 20) - 1, 1 << 20, n - 257, n - 2, n - 1], device="cuda")
    for name in ("mxfp8", "mxfp4"):
        r = q.rmsnorm(x, w, quant=act(q, name))
        small = q.rmsnorm(x[at].contiguous(), w, quant=act(q, name))
        assert torch.equal(r.codes.view(torch.uint8)[at], small.codes.view(torch.uint8))
        assert torch.equal(r.scale.view(torch.uint8)[at], small.scale.view(torch.uint8))
        xq, xs = getattr(q, f"quantize_{name}")(x)
        assert torch.equal(xq.view(torch.uint8)[at], getattr(q, f"quantize_{name}")(x[at].contiguous())[0].view(torch.uint8))
        assert torch.equal(q.dequant_mx(xq, xs, torch.bfloat16)[at], q.dequant_mx(xq.view(torch.uint8)[at].view(xq.dtype), xs.view(torch.uint8)[at], torch.bfloat16))
        y = q.gemm_mxfp4(wq, ws, xq, xs, dtype=torch.bfloat16)
        check(y[at], wide(wq, ws), wide(xq.view(torch.uint8)[at].view(xq.dtype), xs.view(torch.uint8)[at]), name)
        y2 = q.linear_mxfp4(x, wq, ws, act=act(q, name))
        assert torch.equal(y, y2)
