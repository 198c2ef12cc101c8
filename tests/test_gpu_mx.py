"""The microscaling formats, their products and the norm with quantized output on
the GPU, against plain 64-bit forms.

Codes and scales of given values: the rule is exact arithmetic, so bytes are equal.

Products: within 2e-5 * sum|w x| of the exact product of the codes where sums are
exact to fp32 rounding (MXFP4 activations; MXFP8 ones with fp32 results): k additions
of at most 2^-24 of the running magnitude, 14336 * 2^-24 = 8.6e-4 at worst in one
chain, but a result is the sum of at least 8 waves' or many instructions' chains
of 32 columns and more, 14336 / 32 * 2^-24 = 2.7e-5, half of it on average over the
chain's length.  16-bit results of MXFP8 activations lose at most 7 * 2^-13 of the
largest product of each 8 columns besides, at most 7 * 2^-13 * sum|w x|.  Then half
a unit of the result's type.

Norm: y in fp32 from t: a thread adds up to 8 V = 32 squares in a chain, then at most
6 + 16 partial sums: 54 roundings of 2^-24 of the sum, half of that after the root;
the division by hidden, eps, the root, its reciprocal and two products 6 more: 33 *
2^-24 of y.  Codes lie between those of y (1 - d) and y (1 + d), d = 2^-18 (64 * 2^-24).
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
HALF_ULP = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 2.0 ** -149, torch.float16: 2.0 ** -24, torch.bfloat16: 2.0 ** -133}
D = 2.0 ** -18
E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
E4M3 = np.array([m * 2.0 ** -9 for m in range(8)] + [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)])[:127]
TABLE = {"mxfp4": (E2M1, 2), "mxfp8": (E4M3, 8)}


@pytest.fixture(scope="module")
def q():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import bit_block_quant_amd as q
    return q


def act(q, name):
    return q.ACTS[name]


def nearest(a, table):
    """Index of the table's value nearest to a >= 0, halves to the even index, the last beyond."""
    a = np.minimum(a, table[-1])
    hi = np.clip(np.searchsorted(table, a), 1, len(table) - 1)
    down, up = a - table[hi - 1], table[hi] - a
    return np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, hi - 1)


def mx_ref(v, name):
    """64-bit values (rows, k) -> code bytes (one per value, with the sign), scale bytes."""
    table, top = TABLE[name]
    t = np.asarray(v, np.float64).reshape(v.shape[0], -1, 32)
    big = np.abs(t).max(-1)
    with np.errstate(all="ignore"):
        _, e = np.frexp(big)
        e = np.where(big == 0, -127, np.maximum(e - 1 - top, -127)).astype(np.int64)
        code = nearest(np.abs(t) / 2.0 ** e[..., None].astype(np.float64), table)
    code = code + np.signbit(t) * (8 if name == "mxfp4" else 128)
    bad = ~np.isfinite(t).all(-1)
    code[bad] = 0
    return code.reshape(v.shape).astype(np.uint8), np.where(bad, 255, e + 127).astype(np.uint8)


def unpack(codes):
    """Code bytes (rows, k) of what the library returns."""
    b = codes.view(torch.uint8).cpu().numpy()
    if codes.dtype != torch.uint8:
        return b
    out = np.empty((b.shape[0], 2 * b.shape[1]), np.uint8)
    out[:, ::2], out[:, 1::2] = b & 15, b >> 4
    return out


def scale_bytes(s):
    return s.view(torch.uint8).cpu().numpy()


def values(code, scale, name):
    table, _ = TABLE[name]
    sign = 8 if name == "mxfp4" else 128
    with np.errstate(all="ignore"):
        v = np.where(code & sign, -1.0, 1.0) * np.append(table, [np.nan] * (sign - len(table)))[code & (sign - 1)]
        s = np.where(scale == 255, np.nan, 2.0 ** (scale.astype(np.float64) - 127))
    return v * np.repeat(s, 32, 1)


def f64(t):
    return t.detach().float().cpu().double().numpy()


def odd_values(rng, rows, k):
    """Rows of several flavours: normal, outliers, zero, constant, tiny, huge, ties, powers of two, signed zeros."""
    x = rng.standard_normal((rows, k)).astype(np.float32)
    for r in range(rows):
        f = r % 9
        if f == 1:
            x[r, r % k] = 300.0
        elif f == 2:
            x[r] = 0.0
        elif f == 3:
            x[r] = -1.5
        elif f == 4:
            x[r] *= np.float32(2.0 ** -14)
        elif f == 5:
            x[r] *= np.float32(3000.0)
        elif f == 6:  # maximum 4: the scale is 1 (e2m1), and quarters are ties
            x[r] = rng.integers(-16, 17, k) / 4.0
            x[r, ::32] = 4.0
        elif f == 7:
            x[r] = 2.0 ** rng.integers(-12, 5, k) * rng.choice([-1, 1], k)
        elif f == 8:
            x[r, : k // 2] = -0.0
    return x


# ------------------------------------------------------------- quantizers
@pytest.mark.parametrize("name", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,k", [(1, 32), (3, 32), (9, 96), (64, 1152), (130, 4096)])
def test_quantize(q, name, dtype, rows, k):
    x = torch.from_numpy(odd_values(np.random.default_rng(rows + k), rows, k)).to(TYPES[dtype]).cuda()
    codes, scale = getattr(q, f"quantize_{name}")(x)
    want, ws = mx_ref(f64(x), name)
    assert scale.dtype == torch.float8_e8m0fnu and scale.shape == (rows, k // 32)
    assert np.array_equal(scale_bytes(scale), ws)
    assert np.array_equal(unpack(codes), want)


@pytest.mark.parametrize("name", ["mxfp4", "mxfp8"])
def test_quantize_extremes(q, name):
    """fp32 from the smallest subnormals to the largest numbers."""
    rng = np.random.default_rng(3)
    x = rng.standard_normal((300, 64)) * 2.0 ** np.linspace(-155, 128, 300)[:, None]
    x = np.clip(x, -3.4e38, 3.4e38).astype(np.float32)
    x[0, 0], x[0, 32] = 2.0 ** -149, -(2.0 ** -149)
    codes, scale = getattr(q, f"quantize_{name}")(torch.from_numpy(x).cuda())
    want, ws = mx_ref(x, name)
    assert np.array_equal(scale_bytes(scale), ws)
    assert np.array_equal(unpack(codes), want)


@pytest.mark.parametrize("name", ["mxfp4", "mxfp8"])
def test_quantize_every_bf16(q, name):
    """All finite bf16 numbers, each as a block's only value and beside the block's maximum."""
    b = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    b = b[torch.isfinite(b.float())]
    x = torch.zeros(b.numel(), 64, dtype=torch.bfloat16)
    x[:, 5], x[:, 32], x[:, 63] = b, 448.0, b
    codes, scale = getattr(q, f"quantize_{name}")(x.cuda())
    want, ws = mx_ref(f64(x), name)
    assert np.array_equal(scale_bytes(scale), ws)
    assert np.array_equal(unpack(codes), want)


@pytest.mark.parametrize("name", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_quantize_nan_and_infinity(q, name, dtype):
    """A block with one is NaN as a whole, the others keep their bytes."""
    x = torch.randn(5, 128).to(TYPES[dtype])
    plain, ps = getattr(q, f"quantize_{name}")(x.cuda())
    x[1, 33], x[2, 0], x[3, 127], x[4, 64:96] = float("nan"), float("inf"), -float("inf"), float("nan")
    codes, scale = getattr(q, f"quantize_{name}")(x.cuda())
    got, s = unpack(codes).reshape(5, 4, 32), scale_bytes(scale)
    hit = np.zeros((5, 4), bool)
    hit[1, 1] = hit[2, 0] = hit[3, 3] = hit[4, 2] = True
    assert np.all(s[hit] == 255) and np.all(got[hit] == 0)
    assert np.array_equal(s[~hit], scale_bytes(ps)[~hit])
    assert np.array_equal(got[~hit], unpack(plain).reshape(5, 4, 32)[~hit])
    back = f64(q.dequant_mx(codes, scale)).reshape(5, 4, 32)
    assert np.all(np.isnan(back[hit])) and np.all(np.isfinite(back[~hit]))


@pytest.mark.parametrize("out", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("name", ["mxfp4", "mxfp8"])
def test_dequant_every_code_and_scale(q, name, out):
    """All codes under all scale bytes: the fp32 value rounded once to the result's type."""
    n = 16 if name == "mxfp4" else 256
    code = np.tile(np.arange(n, dtype=np.uint8), max(1, 32 // n))
    code = np.tile(code, (256, 1))
    scale = np.repeat(np.arange(256, dtype=np.uint8)[:, None], code.shape[1] // 32, 1)
    packed = code[:, ::2] | (code[:, 1::2] << 4) if name == "mxfp4" else code
    ct = torch.from_numpy(packed).cuda()
    ct = ct if name == "mxfp4" else ct.view(torch.float8_e4m3fn)
    got = q.dequant_mx(ct, torch.from_numpy(scale).cuda(), TYPES[out])
    with np.errstate(all="ignore"):
        want = torch.from_numpy(values(code, scale, name).astype(np.float32)).to(TYPES[out])
    assert np.array_equal(f64(got), f64(want), equal_nan=True)


# --------------------------------------------------------------- products
def operands(q, m, k, n, name, seed=0, spread=3.0):
    rng = np.random.default_rng(seed + m + k + n)
    w = rng.standard_normal((m, k)) * np.exp(rng.uniform(-spread, 0, (m, 1)))
    x = rng.standard_normal((n, k))
    x[:, rng.integers(0, k, 3)] *= 20
    x[:, : k // 2] *= 0.125
    w, x = torch.from_numpy(w.astype(np.float32)).cuda(), torch.from_numpy(x.astype(np.float32)).cuda()
    wq, ws = q.quantize_mxfp4(w)
    xq, xs = getattr(q, f"quantize_{name}")(x)
    return wq, ws, xq, xs, x


def rebuilt(codes, scale, name):
    return values(unpack(codes), scale_bytes(scale), name)


def check(y, W, X, name):
    ref, mag = X @ W.T, np.abs(X) @ np.abs(W).T
    drop = 7 * 2.0 ** -13 if name == "mxfp8" and y.dtype != torch.float32 else 0.0
    err = np.abs(f64(y) - ref)
    assert np.all(err <= (2e-5 + drop) * mag + HALF_ULP[y.dtype] * (np.abs(ref) + 2e-5 * mag) + TINY[y.dtype]), \
        f"off by {np.max(err / np.maximum(mag, 1e-30)):.3g} of sum|w x|"


SIZES = [(1, 32, 1), (16, 64, 1), (5, 96, 3), (17, 160, 2), (33, 256, 16), (100, 288, 17), (64, 512, 33), (129, 992, 65),
         (256, 4096, 1), (300, 4096, 4), (96, 11008, 13), (520, 1312, 130), (257, 2048, 257), (700, 544, 300)]


@pytest.mark.parametrize("out", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("name", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("m,k,n", SIZES)
def test_gemm(q, m, k, n, name, out):
    wq, ws, xq, xs, _ = operands(q, m, k, n, name)
    y = q.gemm_mxfp4(wq, ws, xq, xs, dtype=TYPES[out])
    check(y, rebuilt(wq, ws, "mxfp4"), rebuilt(xq, xs, name), name)
    again = q.gemm_mxfp4(wq, ws, xq, xs, dtype=TYPES[out])
    assert torch.equal(y, again)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("name", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("m,k,n", SIZES)
def test_linear(q, m, k, n, name, dtype):
    """The product of the codes that the call makes itself."""
    wq, ws, _, _, x = operands(q, m, k, n, name)
    x = x.to(TYPES[dtype])
    y = q.linear_mxfp4(x, wq, ws, act=act(q, name))
    assert y.dtype == x.dtype and y.shape == (n, m)
    code, s = mx_ref(f64(x), name)
    check(y, rebuilt(wq, ws, "mxfp4"), values(code, s, name), name)


@pytest.mark.parametrize("name", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("n", [1, 20, 70, 200])
def test_scales_far_apart(q, name, n):
    """Blocks whose scales differ by up to 2^60: fp32 sums keep what an fp32 sum keeps."""
    m, k = 70, 704
    rng = np.random.default_rng(n)
    w = rng.standard_normal((m, k)) * 2.0 ** np.repeat(rng.integers(-30, 30, (m, k // 32)), 32, 1)
    x = rng.standard_normal((n, k)) * 2.0 ** np.repeat(rng.integers(-30, 30, (n, k // 32)), 32, 1)
    wq, ws = q.quantize_mxfp4(torch.from_numpy(w.astype(np.float32)).cuda())
    xq, xs = getattr(q, f"quantize_{name}")(torch.from_numpy(x.astype(np.float32)).cuda())
    check(q.gemm_mxfp4(wq, ws, xq, xs), rebuilt(wq, ws, "mxfp4"), rebuilt(xq, xs, name), name)


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("name", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("m,k,n", [(40, 288, 3), (40, 320, 40), (300, 800, 150)])
def test_nan_stays_in_its_row_and_token(q, m, k, n, name, out):
    wq, ws, xq, xs, _ = operands(q, m, k, n, name)
    plain = q.gemm_mxfp4(wq, ws, xq, xs, dtype=TYPES[out])
    ws, xs = ws.clone(), xs.clone()
    ws.view(torch.uint8)[m - 1, k // 32 - 1] = 255  # the last block of the last row
    ws.view(torch.uint8)[3, 0] = 255
    xs.view(torch.uint8)[n - 1, k // 32 - 1] = 255
    y = q.gemm_mxfp4(wq, ws, xq, xs, dtype=TYPES[out])
    assert torch.isnan(y[:, 3]).all() and torch.isnan(y[:, m - 1]).all() and torch.isnan(y[n - 1]).all()
    keep = [r for r in range(m) if r not in (3, m - 1)]
    assert torch.equal(y[: n - 1][:, keep], plain[: n - 1][:, keep])


@pytest.mark.parametrize("name", ["mxfp4", "mxfp8"])
def test_zeros_and_empty(q, name):
    wq, ws, xq, xs, x = operands(q, 48, 128, 5, name)
    z, zs = getattr(q, f"quantize_{name}")(torch.zeros(5, 128, device="cuda"))
    assert torch.equal(q.gemm_mxfp4(wq, ws, z, zs), torch.zeros(5, 48, device="cuda"))
    e8 = torch.float8_e8m0fnu
    nothing = torch.empty(0, 0, dtype=e8, device="cuda")
    y = q.gemm_mxfp4(torch.empty(48, 0, dtype=torch.uint8, device="cuda"), nothing,
                     torch.empty(5, 0, dtype=xq.dtype, device="cuda"), nothing, dtype=torch.float16)
    assert torch.equal(y, torch.zeros(5, 48, device="cuda", dtype=torch.float16))
    assert q.gemm_mxfp4(wq, ws, xq[:0], xs[:0]).shape == (0, 48)
    assert q.linear_mxfp4(x[:0], wq, ws, act=act(q, name)).shape == (0, 48)
    assert q.linear_mxfp4(x, wq[:0], ws[:0], act=act(q, name)).shape == (5, 0)
    assert q.dequant_mx(xq[:0], xs[:0]).shape == (0, 128)
    assert getattr(q, f"quantize_{name}")(x[:0])[0].shape[0] == 0


@pytest.mark.parametrize("name", ["mxfp4", "mxfp8"])
def test_rows_of_larger_tensors(q, name):
    """Slices of rows: scales then start at any byte."""
    wq, ws, xq, xs, x = operands(q, 90, 96, 40, name)
    full = q.gemm_mxfp4(wq, ws, xq, xs)
    for a, b, t in [(1, 90, 1), (7, 23, 3), (89, 90, 39)]:
        got = q.gemm_mxfp4(wq[a:b], ws[a:b], xq[t:], xs[t:])
        check(got, rebuilt(wq[a:b], ws[a:b], "mxfp4"), rebuilt(xq[t:], xs[t:], name), name)
        assert torch.allclose(got, full[t:, a:b], rtol=1e-4, atol=1e-3)
    assert torch.equal(q.dequant_mx(xq[3:], xs[3:]), q.dequant_mx(xq, xs)[3:])


# ------------------------------------------------------------------- norm
def norm_ref(x, w, residual, eps, dtype):
    """64-bit y, and t as the type holds it."""
    t = x if residual is None else torch.from_numpy((f64(x) + f64(residual)).astype(np.float32)).to(dtype)
    t64 = f64(t)
    rms = np.sqrt((t64 ** 2).mean(-1, keepdims=True) + eps)
    return t64 / rms * f64(w), t


def between(code, lo, hi):
    assert np.all((code >= np.minimum(lo, hi)) & (code <= np.maximum(lo, hi)))


def check_codes(r, y, quant):
    """Codes and scales of a norm against its 64-bit y."""
    if quant in ("mxfp4", "mxfp8"):
        table, top = TABLE[quant]
        big = np.abs(y).reshape(y.shape[0], -1, 32).max(-1)
        s = scale_bytes(r.scale).astype(np.int64)
        lo, hi = (np.where(big == 0, 0, np.maximum(np.frexp(big * f)[1] + 126 - top, 0)) for f in (1 - D, 1 + D))
        assert np.all((s == lo) | (s == hi))
        got = values(unpack(r.codes), s.astype(np.uint8), quant)
        step = np.repeat(2.0 ** (s - 127.0), 32, 1)
        a, b = (np.sign(y) * table[nearest(np.abs(y) * f / step, table)] * step for f in (1 - D, 1 + D))
        between(got, a, b)
        return
    if quant == "f8":
        big = np.abs(y).reshape(y.shape[0], -1, 128).max(-1)
        s = r.scale.cpu().double().numpy()
        assert np.all(np.abs(s - big / 448) <= 2 * D * big / 448)
        step = np.repeat(s, 128, 1)
        c = r.codes.view(torch.uint8).cpu().numpy()
        got = np.where(c & 128, -1.0, 1.0) * np.append(E4M3, [np.nan])[c & 127]
        with np.errstate(all="ignore"):
            u = np.where(step == 0, 0, y / step)
        a, b = (np.sign(u) * E4M3[nearest(np.abs(u) * f, E4M3)] for f in (1 - 2 * D, 1 + 2 * D))
        between(got, a, b)
        return
    big = np.abs(y).max(-1)
    s = r.scale.cpu().double().numpy()
    assert np.all(np.abs(s - big / 127) <= 2 * D * big / 127)
    with np.errstate(all="ignore"):
        u = np.where(s[:, None] == 0, 0, y / s[:, None])
    half = lambda v: np.sign(v) * np.floor(np.abs(v) + 0.5)  # noqa: E731
    a, b = (np.clip(half(u * f), -127, 127) for f in (1 - 2 * D, 1 + 2 * D))
    between(r.codes.cpu().numpy(), a, b)


NORM = [(1, 128), (3, 384), (5, 512), (2, 640), (7, 4096), (130, 4096), (9, 5120), (4, 11008), (3, 20480), (2, 33024)]


@pytest.mark.parametrize("quant", ["f8", "i8", "mxfp8", "mxfp4"])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("n,h", NORM)
@pytest.mark.parametrize("with_residual", [True, False])
def test_rmsnorm(q, n, h, dtype, quant, with_residual):
    rng = np.random.default_rng(n + h)
    x = torch.from_numpy(odd_values(rng, n, h)).to(TYPES[dtype]).cuda()
    res = torch.from_numpy(rng.standard_normal((n, h)).astype(np.float32)).to(TYPES[dtype]).cuda() if with_residual else None
    w = torch.from_numpy((1 + 0.3 * rng.standard_normal(h)).astype(np.float32)).cuda()
    w = w.to(TYPES[["f32", "f16", "bf16"][(n + h // 128) % 3]])
    r = q.rmsnorm(x, w, res, eps=1e-5, quant=act(q, quant), y=True)
    y, t = norm_ref(x, w, res, 1e-5, TYPES[dtype])
    if with_residual:
        assert torch.equal(r.total.cpu(), t.cpu())
    else:
        assert r.total is None
    assert np.all(np.abs(f64(r.y) - y) <= (D + HALF_ULP[r.y.dtype]) * np.abs(y) + TINY[r.y.dtype])
    check_codes(r, y, quant)
    plain = q.rmsnorm(x, w, res, eps=1e-5, quant=None)
    assert torch.equal(plain.y, r.y) and plain.codes is None and plain.scale is None


@pytest.mark.parametrize("h", [32, 96, 160, 2080])
@pytest.mark.parametrize("quant", ["mxfp8", "mxfp4"])
def test_rmsnorm_ragged_blocks(q, h, quant):
    """Widths that are multiples of 32 only, and of 8 only without codes or with one scale a row."""
    for n in (1, 5, 64):
        x = torch.randn(n, h, device="cuda", dtype=torch.bfloat16)
        w = torch.rand(h, device="cuda") + 0.5
        r = q.rmsnorm(x, w, quant=act(q, quant))
        check_codes(r, norm_ref(x, w, None, 1e-6, x.dtype)[0], quant)
        x8, w8 = x[:, : h - 24].contiguous(), w[: h - 24].contiguous()
        check_codes(q.rmsnorm(x8, w8, quant=q.ACT_I8), norm_ref(x8, w8, None, 1e-6, x.dtype)[0], "i8")


@pytest.mark.parametrize("quant", ["f8", "i8", "mxfp8", "mxfp4"])
def test_rmsnorm_zero_and_nan_rows(q, quant):
    """A row of zeros gives zeros; a NaN or an infinity stays in its row."""
    x = torch.randn(6, 256, device="cuda", dtype=torch.bfloat16)
    w = torch.ones(256, device="cuda")
    clean = q.rmsnorm(x, w, quant=act(q, quant))
    x[1] = 0
    x[3, 7] = float("nan")
    x[4, 200] = float("inf")
    r = q.rmsnorm(x, w, quant=act(q, quant), y=True)
    assert torch.all(r.y[1] == 0) and torch.isnan(r.y[3]).all() and torch.isnan(r.y[4, 200])
    assert torch.all(r.codes[1].view(torch.uint8) == 0)
    s = r.scale.float().view(6, -1)
    assert torch.isnan(s[3]).all() and torch.isnan(s[4]).any()
    for i in (0, 2, 5):
        assert torch.equal(r.codes[i].view(torch.uint8), clean.codes[i].view(torch.uint8))
        assert torch.equal(s[i], clean.scale.float().view(6, -1)[i])
    y = q.rmsnorm(x[1:2], w, eps=0.0, quant=None).y
    assert torch.isnan(y).all()  # 0 / 0, as the formula has it


def test_rmsnorm_in_place(q):
    """The sum may replace x or the residual."""
    for n, h in ((3, 256), (2, 33024)):
        x, res = (torch.randn(n, h, device="cuda", dtype=torch.float16) for _ in range(2))
        w = torch.rand(h, device="cuda", dtype=torch.float16)
        want = q.rmsnorm(x, w, res, quant=q.ACT_MXFP4)
        for target in (x.clone(), res.clone()):
            a = target if torch.equal(target, x) else x
            b = target if a is not target else res
            got = q.rmsnorm(a, w, b, quant=q.ACT_MXFP4, total=target)
            assert got.total is target and torch.equal(target, want.total)
            assert torch.equal(got.codes, want.codes)


# --------------------------------------------------------------- together
def layer(q, x, res, weights, out=None):
    """What a decoder does before its attention: the norm in every product's own codes, and the products."""
    w, wq, ws, fq, fs, blocks, h = weights
    m = wq.shape[0]
    a = q.rmsnorm(x, w, res, quant=q.ACT_MXFP8)
    b = q.rmsnorm(x, w, res, quant=q.ACT_MXFP4)
    c = q.rmsnorm(x, w, res, quant=q.ACT_F8)
    d = q.rmsnorm(x, w, res, quant=q.ACT_I8)
    return (q.gemm_mxfp4(wq, ws, a.codes, a.scale, dtype=x.dtype), q.gemm_mxfp4(wq, ws, b.codes, b.scale),
            q.gemm_f8(fq, fs, c.codes, c.scale), q.gemm_w4a8(blocks, m, h, d.codes, d.scale), a.total)


@pytest.fixture(scope="module")
def weights(q):
    m, h = 192, 512
    full = torch.randn(m, h, device="cuda") * 0.05
    w = 1 + 0.1 * torch.randn(h, device="cuda")
    return (w, *q.quantize_mxfp4(full), *q.quantize_f8(full), q.quantize(full, q.W4G128), h), full


@pytest.mark.parametrize("n", [1, 6, 40, 150])
def test_norm_and_products(q, weights, n):
    """Each chain stays near the same in fp32.  Relative 2-norm of what rounding x to a format moves:
    e4m3 2^-5, int8 of normal rows 2^-6, e2m1 2^-2 (half a step of at most 1/2 of the value,
    uniform: 2^-2 / sqrt 3 and what saturates), and of the weights' own format as much (4 bits
    with an fp16 scale per 128: 2^-2.5)."""
    parts, full = weights
    x, res = (torch.randn(n, 512, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    y8, y4, f8, i8, total = layer(q, x, res, parts)
    want = f64(torch.from_numpy(norm_ref(x, parts[0], res, 1e-6, x.dtype)[0])) @ f64(full).T
    assert torch.equal(total, (x.float() + res.float()).bfloat16())
    for got, tol in ((y8, 2.0 ** -2), (y4, 2.0 ** -1), (f8, 2.0 ** -4), (i8, 2.0 ** -2)):
        assert np.linalg.norm(f64(got) - want) < tol * np.linalg.norm(want)


@pytest.mark.parametrize("n", [1, 6, 40, 150])
def test_captured_and_replayed(q, weights, n):
    """Norms and products in a graph, replayed on changing inputs with eager work between (the
    int8 product adds its partial sums with atomics unless told not to)."""
    parts, _ = weights
    q.set_deterministic(True)
    try:
        capture_and_replay(q, parts, n)
    finally:
        q.set_deterministic(False)


def capture_and_replay(q, parts, n):
    x, res = (torch.randn(n, 512, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer(q, x, res, parts)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = layer(q, x, res, parts)
    for _ in range(3):
        x.normal_()
        res.normal_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, layer(q, x, res, parts)):
            assert torch.equal(a, b)


def test_two_streams(q, weights):
    """Calls on two streams at once, each with memory of its own."""
    parts, _ = weights
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    xs = [torch.randn(n, 512, device="cuda", dtype=torch.bfloat16) for n in (150, 33)]
    wq, ws = parts[1], parts[2]
    want = [q.linear_mxfp4(x, wq, ws) for x in xs]
    norms = [q.rmsnorm(x, parts[0], x, quant=q.ACT_MXFP8) for x in xs]
    torch.cuda.synchronize()
    got, gn = [], []
    for _ in range(5):
        for x, s in zip(xs, (a, b)):
            got.append(q.linear_mxfp4(x, wq, ws, stream=s))
            gn.append(q.rmsnorm(x, parts[0], x, quant=q.ACT_MXFP8, stream=s))
    torch.cuda.synchronize()
    for i, (g, r) in enumerate(zip(got, gn)):
        assert torch.equal(g, want[i % 2]) and torch.equal(r.total, norms[i % 2].total)
        assert torch.equal(r.codes.view(torch.uint8), norms[i % 2].codes.view(torch.uint8))
