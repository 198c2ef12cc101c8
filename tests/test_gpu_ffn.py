"""The feed-forward operators on the GPU against plain 64-bit forms.

8-bit products (e4m3 codes, a scale for each block of 128): the codes and
scales must equal the definition's bit for bit, the products lie within
2e-5 * sum|w x| of the exact product of the codes (the library's bound) up to
64 tokens, and within 2^-12 * sum|w x| beyond, where the fp8 matrix
instructions keep a group's sum to 2^-13 of its magnitudes at worst.

Mixture of experts: routing must equal a stable sort's, and Y lies within what
the products' bound carries through the formula, plus the 16 mantissa bits of
the intermediate, plus the rounding of the output type.
"""
import ctypes
import math

import numpy as np
import pytest

import oracle as O

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

TOL = 2e-5
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
# half a unit in the last place, relative
HALF_ULP = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}


@pytest.fixture(scope="module")
def q():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import bit_block_quant_amd as q
    return q


def f64(t):
    torch.cuda.synchronize()
    return t.detach().cpu().double().numpy()


# ------------------------------------------------------- e4m3, plainly
def e4m3_table():
    v = np.full(256, np.nan)
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        if e == 15 and m == 7:
            continue
        a = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        v[b] = -a if b & 128 else a
    return v


E4M3 = e4m3_table()
POSITIVE = E4M3[:127]  # 0 .. 448, ascending


def e4m3_round(v):
    """Nearest e4m3 value of |v| <= 448 by search, ties to the even code; codes >= 0."""
    a = np.abs(v)
    hi = np.clip(np.searchsorted(POSITIVE, a), 1, 126)
    lo = hi - 1
    dl, dh = a - POSITIVE[lo], POSITIVE[hi] - a
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    return code


def quant_ref(groups):
    """(..., 128) fp32 values sharing a scale along the last axis -> code magnitudes, signs' values, scales."""
    with np.errstate(divide="ignore", invalid="ignore", over="ignore"):
        s = (np.abs(groups).max(-1, keepdims=True).astype(np.float32) / np.float32(448)).astype(np.float32)
        quot = np.where(s == 0, np.float32(0), groups.astype(np.float32) / s).astype(np.float32)
    quot = np.clip(quot.astype(np.float64), -448, 448)
    return np.sign(quot) * POSITIVE[e4m3_round(quot)], s[..., 0]


def act_ref(x):
    v, s = quant_ref(x.reshape(x.shape[0], -1, 128))
    return v.reshape(x.shape), s


def weight_ref(w):
    rows, k = w.shape
    nb = -(-rows // 128)
    p = np.zeros((nb * 128, k), np.float32)
    p[:rows] = w
    t = p.reshape(nb, 128, k // 128, 128).transpose(0, 2, 1, 3).reshape(nb, k // 128, 128 * 128)
    v, s = quant_ref(t)
    v = v.reshape(nb, k // 128, 128, 128).transpose(0, 2, 1, 3).reshape(nb * 128, k)[:rows]
    return v, s


def values(codes):
    torch.cuda.synchronize()
    return E4M3[codes.view(torch.uint8).cpu().numpy()]


def rebuilt(codes, scale, block_rows):
    v = values(codes)
    s = scale.cpu().double().numpy().reshape(-1, v.shape[1] // 128)
    return v * np.repeat(np.repeat(s, block_rows, 0)[: v.shape[0]], 128, 1)


def odd_values(rng, rows, k):
    """Rows of several flavours: normal, with an outlier, zero, constant, tiny, huge, exact ties."""
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
            x[r] *= np.float32(1e-6)
        elif f == 5:
            x[r] *= np.float32(2000.0)
        elif f == 6:  # maximum 448: the scale is 1 and every half step is a tie
            steps = POSITIVE[rng.integers(0, 126, k)]
            x[r] = (steps + POSITIVE[np.searchsorted(POSITIVE, steps) + 1]) / 2 * rng.choice([-1, 1], k)
            x[r, ::128] = 448.0
        elif f == 7:
            x[r, : k // 2] = 0.0
    return x


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("n,k", [(1, 128), (9, 128), (7, 384), (64, 1152), (130, 256)])
def test_quantize_act_f8(q, dtype, n, k):
    x = torch.from_numpy(odd_values(np.random.default_rng(n + k), n, k)).to(TYPES[dtype]).cuda()
    codes, scale = q.quantize_act_f8(x)
    v, s = act_ref(x.float().cpu().numpy())
    assert codes.dtype == torch.float8_e4m3fn and scale.shape == (n, k // 128)
    assert np.array_equal(scale.cpu().numpy(), s)
    assert np.array_equal(values(codes), v)


def test_quantize_act_f8_extremes(q):
    """Scales outside 2^+-60, subnormal scales and scales that round to zero."""
    rng = np.random.default_rng(3)
    x = rng.standard_normal((12, 256)).astype(np.float32)
    for r, f in enumerate((1e30, 1e25, 1e-20, 1e-30, 1e-36, 1e-38, 1e-40, 1e-43, 7e38 / 8, 1.0, 2.0 ** 61, 2.0 ** -70)):
        x[r] = np.float32(1.0) * x[r] * np.float32(f)
    x = np.clip(x, -3e38, 3e38)
    codes, scale = q.quantize_act_f8(torch.from_numpy(x).cuda())
    v, s = act_ref(x)
    assert np.array_equal(scale.cpu().numpy(), s)
    assert np.array_equal(values(codes), v)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,k", [(1, 128), (127, 256), (128, 128), (130, 384), (300, 640)])
def test_quantize_f8(q, dtype, rows, k):
    w = torch.from_numpy(odd_values(np.random.default_rng(rows), rows, k)).to(TYPES[dtype]).cuda()
    codes, scale = q.quantize_f8(w)
    v, s = weight_ref(w.float().cpu().numpy())
    assert np.array_equal(scale.cpu().numpy(), s)
    assert np.array_equal(values(codes), v)


def f8_operands(q, m, k, n, seed):
    rng = np.random.default_rng(seed)
    w = rng.standard_normal((m, k)).astype(np.float32) * np.exp(rng.uniform(-3, 0, (m, 1))).astype(np.float32)
    x = rng.standard_normal((n, k)).astype(np.float32)
    x[:, rng.integers(0, k, 3)] *= 20
    wq, ws = q.quantize_f8(torch.from_numpy(w).cuda())
    xq, xs = q.quantize_act_f8(torch.from_numpy(x).cuda())
    return wq, ws, xq, xs, torch.from_numpy(x).cuda()


def product_bound(n):
    return TOL if n <= 64 else 2.0 ** -12


def check_product(y, W, X, n):
    ref, mag = X @ W.T, np.abs(X) @ np.abs(W).T
    got = f64(y)
    assert np.all(np.abs(got - ref) <= product_bound(n) * mag + 2 * HALF_ULP[y.dtype] * np.abs(ref) + 1e-38)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_f8_of_nan_and_infinity(q, dtype):
    """A NaN or an infinity shows in its group's scale or codes, and nowhere else."""
    x = torch.randn(5, 384, device="cuda").to(TYPES[dtype])
    plain, scale = q.quantize_act_f8(x)
    x[1, 130] = float("nan")
    x[2, 0] = float("inf")
    x[3, 383] = -float("inf")
    x[4, 256:] = float("nan")
    got, s = q.quantize_act_f8(x)
    s, c = s.cpu(), got.float().cpu()
    assert torch.isnan(s[1, 1]) and torch.isnan(s[4, 2]) and torch.isinf(s[2, 0]) and torch.isinf(s[3, 2])
    assert torch.isnan(c[2, 0]) and torch.all(c[2, 1:128] == 0) and torch.isnan(c[3, 383])
    for t, g in [(1, 1), (2, 0), (3, 2), (4, 2)]:
        keep = [i for i in range(3) if i != g]
        assert torch.equal(s[t, keep], scale.cpu()[t, keep])
        cols = torch.cat([torch.arange(128 * i, 128 * i + 128) for i in keep])
        assert torch.equal(c[t, cols], plain.float().cpu()[t, cols])
    w = torch.randn(256, 384, device="cuda").to(TYPES[dtype])
    w[200, 7] = float("nan")
    _, ws = q.quantize_f8(w)
    assert torch.isnan(ws).sum() == 1 and torch.isnan(ws[1, 0])


@pytest.mark.parametrize("n", [3, 9, 40, 100, 300])
@pytest.mark.parametrize("bad", ["nan", "inf", "-inf"])
def test_f8_products_of_nan(q, n, bad):
    """Every result of a token with a NaN or an infinity is NaN, every other token's is as without."""
    rng = np.random.default_rng(n)
    wq, ws, _, _, x = f8_operands(q, 300, 2048, n, n)
    w13, s13, _, _, _ = f8_operands(q, 512, 2048, 1, n)
    w2, s2, _, _, _ = f8_operands(q, 2048, 256, 1, n)
    keep = torch.arange(n, device="cuda") != n // 2
    for dtype in (torch.float32, torch.bfloat16):
        x = x.to(dtype)
        poisoned = x.clone()
        poisoned[n // 2, 1000] = float(bad)
        for call in (lambda v: q.linear_f8(v, wq, ws), lambda v: q.ffn_f8(v, w13, s13, w2, s2)):
            y, z = call(x), call(poisoned)
            assert torch.equal(y[keep], z[keep]) and torch.isnan(z[n // 2]).all()


SIZES = [(1, 128, 1), (16, 128, 3), (100, 384, 2), (257, 1152, 5), (128, 4224, 16), (48, 256, 17), (272, 384, 33),
         (1000, 640, 64), (100, 128, 65), (256, 384, 100), (300, 1152, 129), (257, 256, 300), (640, 2176, 257),
         (515, 128, 700), (1024, 1024, 1024)]


@pytest.mark.parametrize("m,k,n", SIZES)
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_gemm_f8(q, m, k, n, dtype):
    wq, ws, xq, xs, _ = f8_operands(q, m, k, n, m + k + n)
    y = q.gemm_f8(wq, ws, xq, xs, dtype=TYPES[dtype])
    assert y.shape == (n, m) and y.dtype == TYPES[dtype]
    check_product(y, rebuilt(wq, ws, 128), rebuilt(xq, xs, 1), n)


@pytest.mark.parametrize("m,k,n", SIZES)
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_linear_f8_is_quantize_and_gemm(q, m, k, n, dtype):
    wq, ws, _, _, x = f8_operands(q, m, k, n, m + k)
    x = x.to(TYPES[dtype])
    y = q.linear_f8(x, wq, ws, dtype=torch.float32)
    xq, xs = q.quantize_act_f8(x)
    assert torch.equal(y, q.gemm_f8(wq, ws, xq, xs))
    assert q.linear_f8(x, wq, ws).dtype == x.dtype


def test_gemm_f8_codes_of_all_magnitudes(q):
    """Every finite code in both operands, scales far apart; up to 64 tokens the sums are fp32."""
    rng = np.random.default_rng(8)
    codes = np.array([b for b in range(256) if not np.isnan(E4M3[b])], np.uint8)
    for n in (5, 64):
        wq = torch.from_numpy(rng.choice(codes, (130, 512))).cuda()
        xq = torch.from_numpy(rng.choice(codes, (n, 512))).cuda()
        ws = torch.from_numpy(np.exp2(rng.uniform(-30, 30, (2, 4))).astype(np.float32)).cuda()
        xs = torch.from_numpy(np.exp2(rng.uniform(-30, 30, (n, 4))).astype(np.float32)).cuda()
        check_product(q.gemm_f8(wq, ws, xq, xs), rebuilt(wq, ws, 128), rebuilt(xq, xs, 1), n)


@pytest.mark.parametrize("n", [1, 3, 40, 200])
def test_gemm_f8_reproducible_and_row_by_row(q, n):
    """Equal bits in repeated calls, and a token's row does not depend on the other tokens' values."""
    wq, ws, xq, xs, _ = f8_operands(q, 300, 1152, n, n)
    y = q.gemm_f8(wq, ws, xq, xs)
    assert torch.equal(y, q.gemm_f8(wq, ws, xq, xs))
    bad = xs.clone()
    bad[n // 2] = float("nan")
    z = q.gemm_f8(wq, ws, xq, bad)
    keep = torch.arange(n, device="cuda") != n // 2
    assert torch.equal(y[keep], z[keep]) and torch.isnan(z[n // 2]).all()


def silu_ref(g):
    return g / (1.0 + np.exp(-np.clip(g, -700, None)))


@pytest.mark.parametrize("hidden,inter,n", [(128, 128, 1), (256, 640, 2), (384, 256, 5), (512, 384, 16), (128, 256, 40),
                                            (256, 384, 64), (384, 256, 65), (512, 640, 300), (256, 128, 513)])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_ffn_f8(q, hidden, inter, n, dtype):
    """A sum that lands on the other side of a tie of the intermediate's codes moves
    one code by a step (at most 1/8 of it).  With the products off by d relative
    to the result, about d * 2^4 of the codes do: for d = 1e-5 that is 2e-4 of
    them, 2e-3 of the result in the 2-norm; 4e-3 leaves room for small sizes."""
    rng = np.random.default_rng(hidden + inter + n)
    x = torch.from_numpy(rng.standard_normal((n, hidden)).astype(np.float32)).to(TYPES[dtype]).cuda()
    w13, s13 = q.quantize_f8(torch.from_numpy(rng.standard_normal((2 * inter, hidden)).astype(np.float32) * 0.1).cuda())
    w2, s2 = q.quantize_f8(torch.from_numpy(rng.standard_normal((hidden, inter)).astype(np.float32) * 0.1).cuda())
    y = q.ffn_f8(x, w13, s13, w2, s2)
    assert y.dtype == x.dtype and y.shape == x.shape
    xv, xsc = act_ref(x.float().cpu().numpy())
    gu = (xv * np.repeat(xsc.astype(np.float64), 128, 1)) @ rebuilt(w13, s13, 128).T
    hv, hs = act_ref((silu_ref(gu[:, :inter]) * gu[:, inter:]).astype(np.float32))
    ref = (hv * np.repeat(hs.astype(np.float64), 128, 1)) @ rebuilt(w2, s2, 128).T
    err = np.linalg.norm(f64(y) - ref) / np.linalg.norm(ref)
    assert err <= 4e-3 + HALF_ULP[x.dtype], err
    assert torch.equal(y, q.ffn_f8(x, w13, s13, w2, s2))


@pytest.mark.parametrize("hidden,inter,n", [(2048, 384, 100), (2048, 14336, 24), (2048, 14336, 64), (1152, 128, 129),
                                            (4096, 128, 65), (1024, 2816, 1600)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_ffn_f8_long_sums(q, hidden, inter, n, dtype):
    """Enough columns for the first product's sums to be split; same bound as above."""
    gen = torch.Generator("cuda").manual_seed(hidden + inter + n)
    x = torch.randn(n, hidden, device="cuda", generator=gen).to(TYPES[dtype])
    w13, s13 = q.quantize_f8(torch.randn(2 * inter, hidden, device="cuda", generator=gen) * 0.1)
    w2, s2 = q.quantize_f8(torch.randn(hidden, inter, device="cuda", generator=gen) * 0.1)
    y = q.ffn_f8(x, w13, s13, w2, s2)
    back = lambda c, s, rows: (torch.from_numpy(E4M3).cuda()[c.view(torch.uint8).long()]
                               * s.double().repeat_interleave(rows, 0)[:c.shape[0]].repeat_interleave(128, 1))
    xv, xsc = act_ref(x.float().cpu().numpy())
    gu = torch.from_numpy(xv * np.repeat(xsc.astype(np.float64), 128, 1)).cuda() @ back(w13, s13, 128).T
    hv, hs = act_ref(f64((gu[:, :inter] / (1 + torch.exp(-gu[:, :inter])) * gu[:, inter:]).float()).astype(np.float32))
    ref = f64(torch.from_numpy(hv * np.repeat(hs.astype(np.float64), 128, 1)).cuda() @ back(w2, s2, 128).T)
    err = np.linalg.norm(f64(y) - ref) / np.linalg.norm(ref)
    assert err <= 4e-3 + HALF_ULP[x.dtype], err
    assert torch.equal(y, q.ffn_f8(x, w13, s13, w2, s2))


@pytest.mark.parametrize("m,k,n", [(9000, 8192, 17), (9000, 8192, 64), (40, 11008, 7), (5000, 11008, 333), (1003, 4096, 70),
                                   (2, 4096, 300), (4097, 8192, 31), (5003, 1024, 4096)])
def test_gemm_f8_large(q, m, k, n):
    """Sizes on the tile kernel's side up to 64 tokens, long sums, many splits."""
    wq, ws, xq, xs, _ = f8_operands(q, m, k, n, 3)
    t = torch.from_numpy(E4M3).cuda()
    W = t[wq.view(torch.uint8).long()] * ws.double().repeat_interleave(128, 0)[:m].repeat_interleave(128, 1)
    X = t[xq.view(torch.uint8).long()] * xs.double().repeat_interleave(128, 1)
    ref, mag = f64(X @ W.T), f64(X.abs() @ W.abs().T)
    for dtype in (torch.float32, torch.bfloat16):
        got = f64(q.gemm_f8(wq, ws, xq, xs, dtype=dtype))
        assert np.all(np.abs(got - ref) <= product_bound(n) * mag + 2 * HALF_ULP[dtype] * np.abs(ref) + 1e-38)


def test_ffn_f8_large_gates(q):
    """Gates far beyond exp's range on both sides: silu is 0 or the gate itself, never NaN."""
    x = torch.ones(3, 128, device="cuda")
    x[1] *= -1
    x[2] = 0
    w13 = torch.ones(256, 128, device="cuda") * 50
    w2 = torch.ones(128, 128, device="cuda")
    (a, sa), (b, sb) = q.quantize_f8(w13), q.quantize_f8(w2)
    y = f64(q.ffn_f8(x, a, sa, b, sb))
    assert np.allclose(y[0], 6400.0 ** 2 * 128, rtol=1e-5) and np.all(y[1:] == 0)


# ----------------------------------------------------- mixture of experts
FMT = {"q4_0": O.Q4_0, "sb4": O.SB4, "sb4_affine": O.SB4_AFFINE, "q4_k": O.Q4_K}


class Layer:
    def __init__(self, q, fmt, experts, hidden, inter, seed):
        rng = np.random.default_rng(seed)
        self.fmt, self.e, self.h, self.i = FMT[fmt], experts, hidden, inter
        spread = np.exp(rng.uniform(-1, 1, (experts, 1, 1))).astype(np.float32)
        up = rng.standard_normal((experts, 2 * inter, hidden)).astype(np.float32) * 0.1 * spread
        down = rng.standard_normal((experts, hidden, inter)).astype(np.float32) * 0.1
        self.gate_up = q.quantize(torch.from_numpy(up.reshape(-1, hidden)).cuda(), self.fmt)
        self.down = q.quantize(torch.from_numpy(down.reshape(-1, inter)).cuda(), self.fmt)
        self.up64 = O.dequant(self.fmt, self.gate_up.cpu().numpy(), 2 * inter * experts, hidden).astype(np.float64).reshape(up.shape)
        self.down64 = O.dequant(self.fmt, self.down.cpu().numpy(), hidden * experts, inter).astype(np.float64).reshape(down.shape)

    def ref(self, x, ids, weights):
        """Y and its bound in 64 bits, from ids (n, k) and weights (n, k)."""
        y = np.zeros((x.shape[0], self.h))
        tol = np.zeros_like(y)
        for t in range(x.shape[0]):
            for e, w in zip(ids[t], weights[t]):
                if not 0 <= e < self.e:
                    continue
                gu, mag = self.up64[e] @ x[t], np.abs(self.up64[e]) @ np.abs(x[t])
                g, u = gu[: self.i], gu[self.i:]
                dg, du = TOL * mag[: self.i], TOL * mag[self.i:]
                s = silu_ref(g)
                h = s * u
                dh = 1.1 * dg * (np.abs(u) + du) + np.abs(s) * du + 2.0 ** -16 * np.abs(h)
                d = np.abs(self.down64[e])
                y[t] += w * (self.down64[e] @ h)
                tol[t] += abs(w) * (d @ (dh + TOL * np.abs(h)))
        return y, tol


def route_ref(logits, top_k, renorm, scale=1.0):
    n, e = logits.shape
    ids = np.full((n, top_k), -1)
    weights = np.zeros((n, top_k))
    for t in range(n):
        row = np.minimum(np.where(np.isnan(logits[t]), -np.inf, logits[t]).astype(np.float64), float(np.finfo(np.float32).max))
        order = [j for j in sorted(range(e), key=lambda j: (-row[j], j)) if row[j] > -np.inf]
        taken = order[:top_k]
        if not taken:
            continue
        p = {j: math.exp(row[j] - row[order[0]]) for j in order}
        total = math.fsum(p[j] for j in (taken if renorm else order))
        ids[t, : len(taken)] = taken
        weights[t, : len(taken)] = [p[j] / total * scale for j in taken]
    return ids, weights


def check_moe(layer, x, y, ids, weights):
    ref, tol = layer.ref(f64(x), ids, weights)
    got = f64(y)
    over = np.abs(got - ref) - (tol + 2 * HALF_ULP[y.dtype] * np.abs(ref))
    assert np.all(over <= 0), (over.max(), np.abs(ref).max())


MOE = [("sb4", 5, 512, 256, 1, 2), ("sb4", 8, 256, 768, 4, 3), ("sb4_affine", 5, 512, 256, 3, 2),
       ("q4_k", 6, 256, 512, 7, 4), ("q4_0", 5, 512, 256, 2, 2), ("q4_0", 4, 96, 160, 5, 2),
       ("q4_0", 3, 32, 32, 1, 1), ("q4_0", 7, 288, 416, 19, 3), ("sb4", 2, 256, 256, 40, 2),
       ("sb4_affine", 70, 256, 256, 9, 8), ("q4_k", 1, 256, 256, 17, 1), ("q4_0", 130, 64, 64, 16, 6),
       ("q4_k", 3, 2304, 256, 6, 2), ("sb4", 3, 256, 2560, 6, 2), ("sb4", 3, 4096, 256, 20, 2),
       ("q4_0", 9, 4128, 96, 33, 3)]


@pytest.mark.parametrize("fmt,experts,hidden,inter,n,top_k", MOE)
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("renorm", [True, False])
def test_moe(q, fmt, experts, hidden, inter, n, top_k, dtype, renorm):
    layer = Layer(q, fmt, experts, hidden, inter, experts + hidden + n)
    rng = np.random.default_rng(n)
    x = torch.from_numpy(rng.standard_normal((n, hidden)).astype(np.float32)).to(TYPES[dtype]).cuda()
    logits = rng.standard_normal((n, experts)).astype(np.float32)
    ids_ref, w_ref = route_ref(logits, top_k, renorm, 1.5)
    for out in (torch.float32, TYPES[dtype]):
        y, ids, weights = q.moe(layer.fmt, x, torch.from_numpy(logits).cuda(), layer.gate_up, layer.down, inter, top_k,
                                renorm=renorm, weight_scale=1.5, dtype=out)
        assert y.dtype == out and y.shape == (n, hidden)
        assert np.array_equal(ids.cpu().numpy(), ids_ref)
        assert np.allclose(f64(weights), w_ref, rtol=2e-6, atol=0)
        check_moe(layer, x, y, ids_ref, f64(weights))


def test_moe_masks_ties_and_extremes(q):
    """Rows that leave fewer than top_k experts, or none; equal logits; NaN, both infinities, the lowest finite value."""
    layer = Layer(q, "sb4", 9, 256, 256, 1)
    inf, nan, low = np.inf, np.nan, np.finfo(np.float32).min
    rows = [[-inf] * 9, [nan] * 9, [-inf] * 4 + [0.5] + [-inf] * 4, [1.0] * 9, [nan, 2, nan, 2, -inf, 2, nan, 1, 1],
            [low] * 9, [-inf, low, -inf, low, low, -inf, low, -inf, low], [inf, 0, 0, inf, 0, 0, 0, 0, 0],
            [3e38, -3e38, 3e38, 0, 0, 0, 0, 0, 0], [0, 1, 2, 3, 4, 5, 6, 7, 8], [-0.0, 0.0, -0.0, 0.0, 0, 0, 0, 0, 0],
            [-200, -100, -100, -300, -101, -150, -100.5, -90, -1000]]
    logits = np.array(rows, np.float32)
    x = torch.from_numpy(np.random.default_rng(2).standard_normal((len(rows), 256)).astype(np.float32)).half().cuda()
    x[0] = float("nan")  # a token that no expert takes is not looked at
    x[1] = float("inf")
    for renorm in (True, False):
        y, ids, weights = q.moe(layer.fmt, x, torch.from_numpy(logits).cuda(), layer.gate_up, layer.down, 256, 4, renorm=renorm)
        ids_ref, w_ref = route_ref(logits, 4, renorm)
        assert np.array_equal(ids.cpu().numpy(), ids_ref)
        assert np.allclose(f64(weights), w_ref, rtol=2e-6, atol=1e-38)
        assert torch.all(y[:2] == 0)
        check_moe(layer, x[2:], y[2:], ids_ref[2:], f64(weights)[2:])


def test_moe_tokens_do_not_mix(q):
    """NaN and infinities in one token, or in an expert's scales, reach only what uses them."""
    layer = Layer(q, "sb4", 6, 256, 256, 4)
    rng = np.random.default_rng(5)
    x = torch.from_numpy(rng.standard_normal((20, 256)).astype(np.float32)).bfloat16().cuda()
    logits = torch.from_numpy(rng.standard_normal((20, 6)).astype(np.float32)).cuda()
    y, ids, _ = q.moe(layer.fmt, x, logits, layer.gate_up, layer.down, 256, 2)
    bad = x.clone()
    bad[3], bad[11] = float("nan"), float("inf")
    z, _, _ = q.moe(layer.fmt, bad, logits, layer.gate_up, layer.down, 256, 2)
    keep = torch.tensor([t not in (3, 11) for t in range(20)], device="cuda")
    assert torch.equal(y[keep], z[keep]) and torch.isnan(z[3]).all()
    for which in ("gate_up", "down"):  # expert 0's first super-scale becomes infinite
        blocks = {"gate_up": layer.gate_up.clone(), "down": layer.down.clone()}
        blocks[which][:2] = torch.tensor([0x00, 0x7C], dtype=torch.uint8, device="cuda")
        z, _, _ = q.moe(layer.fmt, x, logits, blocks["gate_up"], blocks["down"], 256, 2)
        keep = (ids != 0).all(1)
        assert keep.any() and not keep.all() and torch.equal(y[keep], z[keep])


@pytest.mark.parametrize("fmt", ["q4_0", "sb4"])
def test_moe_given_routing(q, fmt):
    """ids and weights of a router of the caller's: repeated experts, ids outside the range, weights of any sign."""
    layer = Layer(q, fmt, 5, 256, 512, 6)
    rng = np.random.default_rng(7)
    ids = rng.integers(-2, 8, (11, 3)).astype(np.int32)
    ids[0], ids[1], ids[2] = -1, [2, 2, 2], [4, 2147483647, -2147483648]
    weights = rng.standard_normal((11, 3)).astype(np.float32)
    weights[(ids < 0) | (ids >= 5)] = np.nan  # never read
    x = torch.from_numpy(rng.standard_normal((11, 256)).astype(np.float32)).half().cuda()
    i, w = torch.from_numpy(ids).cuda(), torch.from_numpy(weights).cuda()
    y, i2, w2 = q.moe(layer.fmt, x, None, layer.gate_up, layer.down, 512, 3, experts=5, ids=i, weights=w, dtype=torch.float32)
    assert np.array_equal(i2.cpu().numpy(), ids) and np.array_equal(w2.cpu().numpy(), weights, equal_nan=True)
    check_moe(layer, x, y, ids, weights.astype(np.float64))


def test_moe_more_pairs_than_one_piece(q):
    """Tokens past one pair of launches: 33 tokens x 32 experts, and 1030 tokens x 1 expert."""
    for experts, top_k, n in ((40, 32, 33), (3, 1, 1030)):
        layer = Layer(q, "q4_0", experts, 64, 32, n)
        rng = np.random.default_rng(n)
        x = torch.from_numpy(rng.standard_normal((n, 64)).astype(np.float32)).half().cuda()
        logits = rng.standard_normal((n, experts)).astype(np.float32)
        y, ids, weights = q.moe(layer.fmt, x, torch.from_numpy(logits).cuda(), layer.gate_up, layer.down, 32, top_k, dtype=torch.float32)
        ids_ref, w_ref = route_ref(logits, top_k, True)
        assert np.array_equal(ids.cpu().numpy(), ids_ref)
        check_moe(layer, x, y, ids_ref, f64(weights))


def test_moe_most_experts(q):
    """512 experts, the most a call takes."""
    layer = Layer(q, "q4_0", 512, 32, 32, 9)
    rng = np.random.default_rng(10)
    x = torch.from_numpy(rng.standard_normal((6, 32)).astype(np.float32)).half().cuda()
    logits = rng.standard_normal((6, 512)).astype(np.float32)
    logits[0] = 0.25
    logits[1, :500] = -np.inf
    y, ids, weights = q.moe(layer.fmt, x, torch.from_numpy(logits).cuda(), layer.gate_up, layer.down, 32, 10, renorm=False, dtype=torch.float32)
    ids_ref, w_ref = route_ref(logits, 10, False)
    assert np.array_equal(ids.cpu().numpy(), ids_ref)
    check_moe(layer, x, y, ids_ref, f64(weights))


# ------------------------------------------------ streams, graphs, bounds
def calls(q):
    """name -> (a function of the output tensors, the outputs)"""
    rng = np.random.default_rng(20)
    out = {}
    for n in (1, 20, 150):
        wq, ws, xq, xs, x = f8_operands(q, 200, 640, n, n)
        y = torch.empty(n, 200, device="cuda")
        out[f"gemm{n}"] = (lambda y=y, a=(wq, ws, xq, xs): q.gemm_f8(*a, out=y), (y,))
        z = torch.empty(n, 200, device="cuda", dtype=torch.bfloat16)
        work = torch.empty(q.lib().qblk_linear_f8_workspace(200, 640, n), dtype=torch.uint8, device="cuda")
        out[f"linear{n}"] = (lambda z=z, a=(x.bfloat16(), wq, ws), work=work: q.linear_f8(*a, out=z, workspace=work), (z,))
        w13, s13, _, _, _ = f8_operands(q, 512, 128, 1, n + 1)
        w2, s2, _, _, xh = f8_operands(q, 128, 256, 1, n + 2)
        v = torch.empty(n, 128, device="cuda", dtype=torch.float16)
        xh = torch.from_numpy(rng.standard_normal((n, 128)).astype(np.float32)).half().cuda()
        work = torch.empty(q.lib().qblk_ffn_f8_workspace(128, 256, n), dtype=torch.uint8, device="cuda")
        out[f"ffn{n}"] = (lambda v=v, a=(xh, w13, s13, w2, s2), work=work: q.ffn_f8(*a, out=v, workspace=work), (v,))
    layer = Layer(q, "sb4", 6, 256, 512, 21)
    for n in (1, 20):
        x = torch.from_numpy(rng.standard_normal((n, 256)).astype(np.float32)).half().cuda()
        logits = torch.from_numpy(rng.standard_normal((n, 6)).astype(np.float32)).cuda()
        y = torch.empty(n, 256, device="cuda", dtype=torch.float16)
        ids, w = torch.empty(n, 2, device="cuda", dtype=torch.int32), torch.empty(n, 2, device="cuda")
        work = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
        out[f"moe{n}"] = (lambda a=(layer.fmt, x, logits, layer.gate_up, layer.down, 512, 2), k=dict(out=y, ids=ids, weights=w, workspace=work):
                          q.moe(*a, **k), (y, ids, w))
    return out


def test_new_memory_belongs_to_the_calls_stream(q, monkeypatch):
    """Results and workspaces that a call allocates come from the pool of the stream it
    runs on: from the current stream's they might be in use there, or be given away
    while the call still runs."""
    side = torch.cuda.Stream()
    made = []
    empty = torch.empty

    def record(*a, **kw):
        made.append(empty(*a, **kw))
        return made[-1]

    wq, ws, xq, xs, x = f8_operands(q, 300, 2048, 70, 1)
    w13, s13, _, _, _ = f8_operands(q, 512, 2048, 1, 1)
    w2, s2, _, _, _ = f8_operands(q, 2048, 256, 1, 1)
    layer = Layer(q, "sb4", 6, 256, 256, 4)
    h, logits = torch.randn(5, 256, device="cuda").half(), torch.randn(5, 6, device="cuda")
    side.wait_stream(torch.cuda.current_stream())
    monkeypatch.setattr(q.torch, "empty", record)
    q.quantize_f8(x, stream=side)
    q.quantize_act_f8(x, stream=side)
    q.gemm_f8(wq, ws, xq, xs, stream=side)
    q.linear_f8(x, wq, ws, stream=side)
    q.ffn_f8(x, w13, s13, w2, s2, stream=side)
    q.moe(layer.fmt, h, logits, layer.gate_up, layer.down, 256, 2, stream=side)
    monkeypatch.undo()
    torch.cuda.synchronize()
    assert len(made) >= 12
    segments = torch.cuda.memory_snapshot()
    for t in made:
        (seg,) = [g for g in segments if g["address"] <= t.data_ptr() < g["address"] + g["total_size"]]
        assert seg["stream"] == side.cuda_stream


def test_other_stream_and_graph(q):
    """The same bits on a stream of the caller's, and from a captured graph at every replay."""
    for name, (call, outs) in calls(q).items():
        call()
        torch.cuda.synchronize()
        want = [o.clone() for o in outs]
        s = torch.cuda.Stream()
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            call()
        s.synchronize()
        assert all(torch.equal(o, w) for o, w in zip(outs, want)), name
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        for _ in range(3):
            for o in outs:
                o.fill_(-7)
            torch.cuda.synchronize()
            g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(o, w) for o, w in zip(outs, want)), name
            torch.randn(1000, device="cuda").sum().item()


MARGIN = 4096


class Padded:
    """A copy of a tensor between margins of 0xFF bytes."""

    def __init__(self, t):
        raw = t.contiguous().view(-1).view(torch.uint8)
        self.n = raw.numel()
        self.whole = torch.full((self.n + 2 * MARGIN,), 0xFF, dtype=torch.uint8, device="cuda")
        self.whole[MARGIN:MARGIN + self.n] = raw
        self.t = self.whole[MARGIN:MARGIN + self.n].view(t.dtype).view(t.shape)

    def intact(self):
        torch.cuda.synchronize()
        w = self.whole.cpu().numpy()
        return bool(np.all(w[:MARGIN] == 0xFF) and np.all(w[MARGIN + self.n:] == 0xFF))


@pytest.mark.parametrize("m,k,n", [(1, 128, 1), (37, 256, 3), (130, 384, 18), (515, 256, 70), (257, 640, 300), (1000, 1152, 513),
                                   (1003, 2048, 70), (254, 2048, 129), (1, 1024, 65), (3, 128, 200)])
def test_f8_bounds(q, m, k, n):
    wq, ws, xq, xs, x = f8_operands(q, m, k, n, 1)
    want = q.gemm_f8(wq, ws, xq, xs)
    pads = [Padded(t) for t in (wq.view(torch.uint8), ws, xq.view(torch.uint8), xs, torch.zeros_like(want))]
    work = Padded(torch.zeros(max(16, q.lib().qblk_gemm_f8_workspace(m, k, n)), dtype=torch.uint8, device="cuda"))
    got = q.gemm_f8(*[p.t for p in pads[:4]], out=pads[4].t, workspace=work.t)
    assert torch.equal(got, want) and all(p.intact() for p in pads + [work])
    for t in (torch.float32, torch.bfloat16):
        px, py = Padded(x.to(t)), Padded(torch.zeros(n, m, dtype=t, device="cuda"))
        work = Padded(torch.zeros(max(16, q.lib().qblk_linear_f8_workspace(m, k, n)), dtype=torch.uint8, device="cuda"))
        got = q.linear_f8(px.t, pads[0].t, pads[1].t, out=py.t, workspace=work.t)
        assert torch.equal(got, q.linear_f8(x.to(t), wq, ws)) and all(p.intact() for p in (px, py, work, *pads))
    pw, pc, psc = Padded(torch.randn(m, k, device="cuda")), Padded(torch.zeros_like(wq.view(torch.uint8))), Padded(torch.zeros_like(ws))
    q.quantize_f8(pw.t, out=pc.t, scale=psc.t)
    assert all(p.intact() for p in (pw, pc, psc))
    px, pc, psc = Padded(x), Padded(torch.zeros_like(xq.view(torch.uint8))), Padded(torch.zeros_like(xs))
    q.quantize_act_f8(px.t, out=pc.t, scale=psc.t)
    assert torch.equal(psc.t, xs) and all(p.intact() for p in (px, pc, psc))


@pytest.mark.parametrize("hidden,inter,n", [(128, 256, 1), (384, 128, 17), (256, 384, 100), (256, 640, 260)])
def test_ffn_f8_bounds(q, hidden, inter, n):
    rng = np.random.default_rng(1)
    w13, s13, _, _, x = f8_operands(q, 2 * inter, hidden, n, 1)
    w2, s2, _, _, _ = f8_operands(q, hidden, inter, 1, 2)
    x = x.bfloat16()
    want = q.ffn_f8(x, w13, s13, w2, s2)
    pads = [Padded(t) for t in (x, w13.view(torch.uint8), s13, w2.view(torch.uint8), s2, torch.zeros_like(want))]
    work = Padded(torch.zeros(q.lib().qblk_ffn_f8_workspace(hidden, inter, n), dtype=torch.uint8, device="cuda"))
    got = q.ffn_f8(*[p.t for p in pads[:5]], out=pads[5].t, workspace=work.t)
    assert torch.equal(got, want) and all(p.intact() for p in pads + [work])


@pytest.mark.parametrize("fmt,experts,hidden,inter,n,top_k", [c for c in MOE if c[4] < 20][:10])
def test_moe_bounds(q, fmt, experts, hidden, inter, n, top_k):
    layer = Layer(q, fmt, experts, hidden, inter, 3)
    rng = np.random.default_rng(4)
    x = torch.from_numpy(rng.standard_normal((n, hidden)).astype(np.float32)).half().cuda()
    logits = torch.from_numpy(rng.standard_normal((n, experts)).astype(np.float32)).cuda()
    y, ids, w = q.moe(layer.fmt, x, logits, layer.gate_up, layer.down, inter, top_k)
    px, pl, pg, pd, py, pi, pw = [Padded(t) for t in (x, logits, layer.gate_up, layer.down, torch.zeros_like(y), torch.zeros_like(ids), torch.zeros_like(w))]
    a = q._Moe(layer.fmt, n, hidden, inter, experts, top_k)
    work = Padded(torch.zeros(q.lib().qblk_moe_workspace(ctypes.byref(a)), dtype=torch.uint8, device="cuda"))
    q.moe(layer.fmt, px.t, pl.t, pg.t, pd.t, inter, top_k, out=py.t, ids=pi.t, weights=pw.t, workspace=work.t)
    assert torch.equal(py.t, y) and torch.equal(pi.t, ids) and torch.equal(pw.t, w)
    assert all(p.intact() for p in (px, pl, pg, pd, py, pi, pw, work))


def test_empty_calls(q):
    e8 = lambda *s: torch.empty(*s, dtype=torch.float8_e4m3fn, device="cuda")  # noqa: E731
    f = lambda *s: torch.empty(*s, device="cuda")  # noqa: E731
    assert q.linear_f8(f(0, 128), e8(5, 128), f(1, 1)).shape == (0, 5)
    assert q.linear_f8(f(3, 128), e8(0, 128), f(0, 1)).shape == (3, 0)
    assert torch.all(q.linear_f8(f(3, 0), e8(5, 0), f(1, 0)) == 0)
    assert torch.all(q.ffn_f8(f(3, 128), e8(0, 128), f(0, 1), e8(128, 0), f(1, 0)) == 0)
    layer = Layer(q, "sb4", 3, 256, 256, 1)
    y, ids, w = q.moe(layer.fmt, f(0, 256).half(), f(0, 3), layer.gate_up, layer.down, 256, 2)
    assert y.shape == (0, 256) and ids.shape == (0, 2) and w.shape == (0, 2)


@pytest.mark.parametrize("hidden,inter", [(256, 0), (0, 256)])
@pytest.mark.parametrize("other", [False, True])
def test_moe_without_columns(q, hidden, inter, other):
    """Nothing is routed: the ids and weights that come back say so, and are not what the memory held."""
    stream = torch.cuda.Stream() if other else None
    x, logits = torch.ones(3, hidden, device="cuda").half(), torch.randn(3, 4, device="cuda")
    none = torch.empty(0, dtype=torch.uint8, device="cuda")
    ids, w = torch.full((3, 2), 7, dtype=torch.int32, device="cuda"), torch.full((3, 2), 7.0, device="cuda")
    torch.cuda.synchronize()
    for given in (dict(ids=ids, weights=w), {}):
        for _ in range(3):  # new memory that held something
            junk = torch.full((3, 2), 5, dtype=torch.int32, device="cuda"), torch.full((3, 2), 5.0, device="cuda")
            del junk
        y, i, v = q.moe(q.SB4, x, logits, none, none, inter, 2, stream=stream, **given)
        torch.cuda.synchronize()
        assert y.shape == (3, hidden) and torch.all(y == 0) and torch.all(i == -1) and torch.all(v == 0)
    ids.fill_(1)
    w.fill_(2.0)
    _, i, v = q.moe(q.SB4, x, None, none, none, inter, 2, experts=4, ids=ids, weights=w)
    assert torch.all(i == 1) and torch.all(v == 2.0)  # a router of the caller's keeps its own
