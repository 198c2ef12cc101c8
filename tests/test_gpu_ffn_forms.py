"""The feed-forward kernels' forms one by one: each tile shape of the 8-bit
products at sizes whose rows, tokens and groups fill nothing evenly, and the
16-row form of the experts' down product (hidden >= 16 rows for every compute
unit) in every format.

Bounds.  fp32 results, at any number of tokens, and all results of up to 64 are
exact to fp32 rounding: 2e-5 * sum|w x|, the library's bound.  16-bit results of
more than 64 tokens: the fp8 matrix instructions bring the products of 8
neighbouring columns to the largest one's exponent and drop what lies below
2^-13 of it, so 7 of them lose less than 7 * 2^-13 of the largest, which is no
more than their sum of magnitudes: 7 * 2^-13 * sum|w x| on any data.

The gated layer's intermediate is quantized again: a sum off by d of its value
moves about d * 2^4 to d * 2^5 of the codes by a step (up to 1/8 of the code).
fp32 sums: d = 3e-7, 1e-5 of the codes, sqrt(1e-5) / 8 = 4e-4 of the result in
the 2-norm; the fp8 instructions' 1e-5 on normal data makes it 1.0e-3 to 2.2e-3.  Beside the
rounding of the result's type (2^-10 / sqrt(12) and 2^-7 / sqrt(12), times 0.72
for significands spread over a binade: 2.0e-4 for f16, 1.6e-3 for bf16): 6e-4
for f32 and f16 results, 3e-3 for bf16.
"""
import ctypes

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from test_gpu_ffn import (E4M3, HALF_ULP, MARGIN, TOL, TYPES, Layer, Padded, act_ref, f64, q,  # noqa: E402, F401
                          route_ref, silu_ref)

pytestmark = pytest.mark.gpu


def wide(codes, scale, rows):
    """Codes and scales (one per `rows` x 128) as float64 values on the GPU."""
    t = torch.from_numpy(E4M3).cuda()
    s = scale.double().view(-1, codes.shape[1] // 128).repeat_interleave(rows, 0)[:codes.shape[0]]
    return t[codes.view(torch.uint8).long()] * s.repeat_interleave(128, 1)


def limit(n, dtype):
    return TOL if n <= 64 or dtype == torch.float32 else 7 * 2.0 ** -13 + TOL


def check_product(y, W, X):
    ref, mag = f64(X @ W.T), f64(X.abs() @ W.abs().T)
    over = np.abs(f64(y) - ref) - (limit(y.shape[0], y.dtype) * mag + HALF_ULP[y.dtype] * 1.01 * np.abs(ref) + 1e-38)
    assert np.all(over <= 0), (over / mag).max()


# ------------------------------------------------------------- 8-bit tiles
# (m, k, n, type): tokens of a tile / 64, whole or K split or rows cut in two launches, on 256 compute units
TILES = [(816, 1152, 1154, "f32"), (416, 1152, 553, "bf16"), (1316, 1152, 2719, "f32"), (1316, 1152, 2719, "bf16"),  # 1, 1, 2, 2
         (2826, 1152, 2719, "f16"),  # 4
         (128, 1152, 66, "f32"), (130, 1152, 67, "bf16"), (555, 6144, 707, "f32"), (1087, 6144, 799, "f16"),  # split: 1, 1, 2, 2
         (5000, 32640, 385, "bf16"),  # split: 4
         (2826, 1152, 2719, "f32"), (33751, 1152, 264, "bf16"),  # cut: 2 and 1
         (3109, 1152, 5013, "bf16"), (2826, 1152, 6402, "f16")]  # cut: 4 and 1, 4 and 2


@pytest.mark.parametrize("m,k,n,dtype", TILES)
def test_tiles(q, m, k, n, dtype):
    gen = torch.Generator("cuda").manual_seed(m + n)
    w = torch.randn(m, k, device="cuda", generator=gen) * torch.exp(-3 * torch.rand(m, 1, device="cuda", generator=gen))
    x = torch.randn(n, k, device="cuda", generator=gen)
    x[:, torch.randint(0, k, (3,), device="cuda", generator=gen)] *= 20
    (wq, ws), (xq, xs) = q.quantize_f8(w), q.quantize_act_f8(x)
    size = n * m * (4 if dtype == "f32" else 2)
    raw = torch.full((size + 2 * MARGIN,), 0xFF, dtype=torch.uint8, device="cuda")
    out = raw[MARGIN:MARGIN + size].view(TYPES[dtype]).view(n, m)
    work = Padded(torch.zeros(max(16, q.lib().qblk_gemm_f8_workspace(m, k, n)), dtype=torch.uint8, device="cuda"))
    y = q.gemm_f8(wq, ws, xq, xs, out=out, workspace=work.t)
    check_product(y, wide(wq, ws, 128), wide(xq, xs, 1))
    assert torch.all(raw[:MARGIN] == 0xFF) and torch.all(raw[MARGIN + size:] == 0xFF) and work.intact()
    assert torch.equal(y, q.gemm_f8(wq, ws, xq, xs, dtype=TYPES[dtype]))


@pytest.mark.parametrize("n", [65, 300])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_codes_of_all_magnitudes_past_64_tokens(q, n, dtype):
    """Every finite code in both operands, so that the products of a group span many binades: the
    16-bit results' bound at its worst, and fp32 results exact to fp32 rounding as ever."""
    rng = np.random.default_rng(n)
    codes = np.array([b for b in range(256) if not np.isnan(E4M3[b])], np.uint8)
    for m, k in ((130, 512), (257, 1152)):
        wq, xq = torch.from_numpy(rng.choice(codes, (m, k))).cuda(), torch.from_numpy(rng.choice(codes, (n, k))).cuda()
        spread = 3 if dtype == "f16" else 30  # (2^-16 * 448^2 * 1152 stays below 65504)
        ws, xs = [torch.from_numpy(np.exp2(rng.uniform(-8 - spread, -8 + spread * (dtype != "f16"), (r, k // 128)))
                                   .astype(np.float32)).cuda() for r in (-(-m // 128), n)]
        check_product(q.gemm_f8(wq, ws, xq, xs, dtype=TYPES[dtype]), wide(wq, ws, 128), wide(xq, xs, 1))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_one_large_product_of_eight(q, dtype):  # noqa: F811
    """Rows of one product of 2^16 and, in the same 8 columns or the next, seven that are 2^-10 to 2^-17 of
    it: what the fp8 instructions drop most of.  fp32 results keep them."""
    x, w = torch.zeros(128, 256, device="cuda"), torch.zeros(128, 256, device="cuda")
    x[:, 0] = w[:, 0] = 256
    for row in range(128):
        e, first = row % 8 - 1, 1 if row < 64 else 8
        x[row, first:first + 7] = [1.0, 1.25, 1.875, -1.875][row // 8 % 4] * 2.0 ** (e // 2)
        w[row, first:first + 7] = [1.0, 1.125, 1.875, 1.875][row // 8 % 4] * 2.0 ** (e - e // 2)
    xs, ws = torch.full((128, 2), 2.0 ** -4, device="cuda"), torch.ones(1, 2, device="cuda")
    wq, xq = w.to(torch.float8_e4m3fn), x.to(torch.float8_e4m3fn)
    assert torch.equal(wq.float(), w) and torch.equal(xq.float(), x)
    check_product(q.gemm_f8(wq, ws, xq, xs, dtype=TYPES[dtype]), wide(wq, ws, 128), wide(xq, xs, 1))


# (hidden, inter, n, type): as above; the split ones join gate and up from partial sums
GATED = [(1152, 384, 1305, "f32"), (1152, 256, 489, "bf16"), (1152, 1408, 1475, "f16"), (1152, 1408, 1475, "bf16"),  # 1, 1, 2, 2
         (1152, 1408, 3100, "bf16"),  # 4
         (1152, 128, 66, "f16"), (1152, 128, 67, "bf16"), (4096, 640, 799, "f32"), (6144, 640, 799, "bf16"),  # split: 1, 1, 2, 2
         (1152, 1408, 3100, "f32"), (1152, 16896, 264, "bf16"),  # cut: 2 and 1
         (1152, 1664, 5013, "bf16"), (1152, 1792, 5665, "bf16")]  # cut: 4 and 1, 4 and 2


@pytest.mark.parametrize("hidden,inter,n,dtype", GATED)
def test_gated_tiles(q, hidden, inter, n, dtype):
    gen = torch.Generator("cuda").manual_seed(inter + n)
    x = torch.randn(n, hidden, device="cuda", generator=gen).to(TYPES[dtype])
    w13, s13 = q.quantize_f8(torch.randn(2 * inter, hidden, device="cuda", generator=gen) * 0.1)
    w2, s2 = q.quantize_f8(torch.randn(hidden, inter, device="cuda", generator=gen) * 0.1)
    xv, xs = act_ref(x.float().cpu().numpy())
    gu = torch.from_numpy(xv * np.repeat(xs.astype(np.float64), 128, 1)).cuda() @ wide(w13, s13, 128).T
    hv, hs = act_ref((gu[:, :inter] / (1 + torch.exp(-gu[:, :inter])) * gu[:, inter:]).float().cpu().numpy())
    ref = torch.from_numpy(hv * np.repeat(hs.astype(np.float64), 128, 1)).cuda() @ wide(w2, s2, 128).T
    work = Padded(torch.zeros(q.lib().qblk_ffn_f8_workspace(hidden, inter, n), dtype=torch.uint8, device="cuda"))
    y = q.ffn_f8(x, w13, s13, w2, s2, workspace=work.t)
    err = ((y.double() - ref).norm() / ref.norm()).item()
    assert err <= (3e-3 if dtype == "bf16" else 6e-4), err
    assert work.intact() and torch.equal(y, q.ffn_f8(x, w13, s13, w2, s2))


# --------------------------------------------- experts, 16 rows a workgroup
HIDDEN, INTER = 4096, 256
FORMATS = ["q4_0", "sb4", "sb4_affine", "q4_k"]


class Wide(Layer):
    def __init__(self, q, fmt, experts, seed):
        super().__init__(q, fmt, experts, HIDDEN, INTER, seed)

    def ref(self, x, ids, weights):
        """As Layer.ref, an expert's tokens at once."""
        y = np.zeros((x.shape[0], self.h))
        tol = np.zeros_like(y)
        for e in range(self.e):
            t, j = np.nonzero(np.asarray(ids) == e)
            if len(t) == 0:
                continue
            w = np.asarray(weights)[t, j][:, None]
            gu, mag = x[t] @ self.up64[e].T, np.abs(x[t]) @ np.abs(self.up64[e]).T
            g, u = gu[:, : self.i], gu[:, self.i:]
            dg, du = TOL * mag[:, : self.i], TOL * mag[:, self.i:]
            s = silu_ref(g)
            h = s * u
            dh = 1.1 * dg * (np.abs(u) + du) + np.abs(s) * du + 2.0 ** -16 * np.abs(h)
            np.add.at(y, t, w * (h @ self.down64[e].T))
            np.add.at(tol, t, np.abs(w) * ((dh + TOL * np.abs(h)) @ np.abs(self.down64[e]).T))
        return y, tol


def check_moe(layer, x, y, ids, weights):
    ref, tol = layer.ref(f64(x), ids, weights)
    over = np.abs(f64(y) - ref) - (tol + 2 * HALF_ULP[y.dtype] * np.abs(ref))
    assert np.all(over <= 0), (over.max(), np.abs(ref).max())


def draw(n, experts, seed, dtype):
    rng = np.random.default_rng(seed)
    x = torch.from_numpy(rng.standard_normal((n, HIDDEN)).astype(np.float32)).to(TYPES[dtype]).cuda()
    logits = rng.standard_normal((n, experts)).astype(np.float32)
    logits[:, 1] += 4.0  # most tokens take expert 1
    return x, logits


@pytest.fixture(scope="module")
def layers(q):  # noqa: F811
    made = {}

    def get(fmt, experts):
        if (fmt, experts) not in made:
            made[fmt, experts] = Wide(q, fmt, experts, 5)
        return made[fmt, experts]
    return get


# one token; more than 16 pairs of one expert; pairs of every slice count; one slice (more than 512 pairs);
# more pairs than one launch takes
@pytest.mark.parametrize("experts,top_k,n", [(4, 2, 1), (4, 2, 20), (16, 8, 5), (4, 3, 90), (4, 2, 300), (4, 2, 520)])
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_moe_16_rows(q, layers, fmt, experts, top_k, n, dtype):  # noqa: F811
    layer = layers(fmt, experts)
    x, logits = draw(n, experts, n, dtype)
    ids_ref, w_ref = route_ref(logits, top_k, True)
    for out in (torch.float32, TYPES[dtype]):
        y, ids, weights = q.moe(layer.fmt, x, torch.from_numpy(logits).cuda(), layer.gate_up, layer.down, INTER, top_k, dtype=out)
        assert np.array_equal(ids.cpu().numpy(), ids_ref)
        assert np.allclose(f64(weights), w_ref, rtol=2e-6, atol=0)
        check_moe(layer, x, y, ids_ref, f64(weights))


@pytest.mark.parametrize("fmt", FORMATS)
def test_moe_16_rows_masks(q, layers, fmt):  # noqa: F811
    """Tokens that leave fewer than top_k experts, or none; a token that no expert takes is not looked at."""
    layer = layers(fmt, 4)
    x, logits = draw(18, 4, 3, "f16")
    logits[:, 2] = -np.inf
    logits[4], logits[5], logits[6] = -np.inf, [np.nan, -np.inf, np.nan, 1.0], np.finfo(np.float32).min
    x[4] = float("nan")
    y, ids, weights = q.moe(layer.fmt, x, torch.from_numpy(logits).cuda(), layer.gate_up, layer.down, INTER, 3, renorm=False)
    ids_ref, w_ref = route_ref(logits, 3, False)
    assert np.array_equal(ids.cpu().numpy(), ids_ref) and np.allclose(f64(weights), w_ref, rtol=2e-6, atol=1e-38)
    keep = np.arange(18) != 4
    assert torch.all(y[4] == 0)
    check_moe(layer, x[keep], y[keep], ids_ref[keep], f64(weights)[keep])


@pytest.mark.parametrize("fmt", FORMATS)
def test_moe_16_rows_tokens_do_not_mix(q, layers, fmt):  # noqa: F811
    layer = layers(fmt, 4)
    x, logits = draw(20, 4, 7, "bf16")
    logits = torch.from_numpy(logits).cuda()
    y, ids, _ = q.moe(layer.fmt, x, logits, layer.gate_up, layer.down, INTER, 2)
    bad = x.clone()
    bad[3], bad[11] = float("nan"), float("inf")
    z, _, _ = q.moe(layer.fmt, bad, logits, layer.gate_up, layer.down, INTER, 2)
    keep = torch.tensor([t not in (3, 11) for t in range(20)], device="cuda")
    assert torch.equal(y[keep], z[keep]) and torch.isnan(z[3]).all()
    for which in ("gate_up", "down"):  # expert 0's first scale becomes infinite
        blocks = {"gate_up": layer.gate_up.clone(), "down": layer.down.clone()}
        blocks[which][:2] = torch.tensor([0x00, 0x7C], dtype=torch.uint8, device="cuda")
        z, _, _ = q.moe(layer.fmt, x, logits, blocks["gate_up"], blocks["down"], INTER, 2)
        keep = (ids != 0).all(1)
        assert keep.any() and not keep.all() and torch.equal(y[keep], z[keep])


@pytest.mark.parametrize("fmt", FORMATS)
def test_moe_16_rows_given_routing(q, layers, fmt):  # noqa: F811
    layer = layers(fmt, 4)
    rng = np.random.default_rng(9)
    ids = rng.integers(-2, 7, (19, 3)).astype(np.int32)
    ids[0], ids[1], ids[2] = -1, [2, 2, 2], [3, 2147483647, -2147483648]
    weights = rng.standard_normal((19, 3)).astype(np.float32)
    weights[(ids < 0) | (ids >= 4)] = np.nan  # never read
    x, _ = draw(19, 4, 11, "f16")
    y, _, _ = q.moe(layer.fmt, x, None, layer.gate_up, layer.down, INTER, 3, experts=4, ids=torch.from_numpy(ids).cuda(),
                    weights=torch.from_numpy(weights).cuda(), dtype=torch.float32)
    check_moe(layer, x, y, ids, weights.astype(np.float64))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("n", [1, 19])
def test_moe_16_rows_bounds_and_graph(q, layers, fmt, n):  # noqa: F811
    """Nothing is written beside the outputs; the same bits from a captured graph at every replay."""
    layer = layers(fmt, 4)
    x, logits = draw(n, 4, 13, "f16")
    logits = torch.from_numpy(logits).cuda()
    want = q.moe(layer.fmt, x, logits, layer.gate_up, layer.down, INTER, 2)
    px, pl, pg, pd, py, pi, pw = [Padded(t) for t in (x, logits, layer.gate_up, layer.down, *[torch.zeros_like(t) for t in want])]
    a = q._Moe(layer.fmt, n, HIDDEN, INTER, 4, 2)
    work = Padded(torch.zeros(q.lib().qblk_moe_workspace(ctypes.byref(a)), dtype=torch.uint8, device="cuda"))

    def call():
        q.moe(layer.fmt, px.t, pl.t, pg.t, pd.t, INTER, 2, out=py.t, ids=pi.t, weights=pw.t, workspace=work.t)
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for replay in range(4):
        if replay:
            py.t.fill_(-7)
            torch.cuda.synchronize()
            g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p.t, w) for p, w in zip((py, pi, pw), want))
        torch.randn(1000, device="cuda").sum().item()
    assert all(p.intact() for p in (px, pl, pg, pd, py, pi, pw, work))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("hidden", [512, HIDDEN])
def test_moe_small_activations(q, fmt, hidden):  # noqa: F811
    """x among the subnormal numbers of f16: its operands keep them."""
    layer = Layer(q, fmt, 3, hidden, 256, 15)
    rng = np.random.default_rng(16)
    x = torch.from_numpy((rng.standard_normal((5, hidden)) * 1e-5).astype(np.float32)).half().cuda()
    logits = rng.standard_normal((5, 3)).astype(np.float32)
    y, ids, weights = q.moe(layer.fmt, x, torch.from_numpy(logits).cuda(), layer.gate_up, layer.down, 256, 2, dtype=torch.float32)
    assert torch.any(y != 0)
    check_moe(layer, x, y, route_ref(logits, 2, True)[0], f64(weights))


def test_moe_largest_intermediate(q):  # noqa: F811
    """1023 pairs of the largest inter, 2^19: their intermediate takes 2 GB, addressed by 32-bit offsets."""
    n, hidden, inter = 1023, 32, 1 << 19
    gen = torch.Generator("cuda").manual_seed(17)
    up, down = [torch.randn(r, c, device="cuda", generator=gen) * s for r, c, s in ((2 * inter, hidden, 0.2), (hidden, inter, 0.01))]
    gate_up, down = q.quantize(up, q.Q4_0), q.quantize(down, q.Q4_0)
    x = torch.randn(n, hidden, device="cuda", generator=gen).half()
    y, _, _ = q.moe(q.Q4_0, x, torch.zeros(n, 1, device="cuda"), gate_up, down, inter, 1, dtype=torch.float32)
    up, down = q.dequant(gate_up, q.Q4_0, 2 * inter, hidden).double(), q.dequant(down, q.Q4_0, hidden, inter).double()
    for t in (0, 1, 500, 1007, 1008, 1022):  # the same formula and bound as above, a token at a time
        v = x[t].double()
        gu, mag = up @ v, up.abs() @ v.abs()
        g, u, dg, du = gu[:inter], gu[inter:], TOL * mag[:inter], TOL * mag[inter:]
        s = g / (1 + torch.exp(-g))
        h = s * u
        dh = 1.1 * dg * (u.abs() + du) + s.abs() * du + 2.0 ** -16 * h.abs()
        tol = down.abs() @ (dh + TOL * h.abs())
        assert torch.all((y[t].double() - down @ h).abs() <= tol + 2.0 ** -23 * (down @ h).abs()), t
