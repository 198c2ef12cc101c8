"""A row's norm is the same whatever rows come with it, and as near to the formula as the
kernel's arithmetic makes it.

The launch takes more threads a row where rows are few, so a row alone and the same row among
a thousand are summed by different threads; their additions pair the same numbers.

y in fp32, in units of u = 2^-24, relative: eight squares in a chain of fused additions put at
most 8 u into a row's sum (all terms have one sign) and 4 u into its root; what is added up
behind that, the division, eps and the root are in 64 bits, the root's reciprocal kept to 2^-46.
t * weight is one rounding (none for 16-bit t and weights), the product with the root's two
parts at most 2 more: 7 u, or 6 u.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from test_gpu_mx import E2M1, E4M3, TYPES, act, q  # noqa: E402, F401

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
# one wave a row up to rows wider than any form holds in registers
WIDTHS = [512, 2048, 2176, 4096, 4224, 8192, 8320, 11008, 16384, 16512, 32768, 33024]


def rows(n, h, dtype, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    x = torch.randn(n, h, device="cuda", generator=gen) * torch.exp(torch.randn(n, 1, device="cuda", generator=gen))
    return x.to(TYPES[dtype])


@pytest.mark.parametrize("with_residual", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("h", WIDTHS)
def test_rows_do_not_see_each_other(q, h, dtype, with_residual):  # noqa: F811
    x = rows(1100, h, dtype, h)  # more rows than four times the compute units, more than them, one
    res = rows(1100, h, dtype, h + 1) if with_residual else None
    w = rows(1, h, "f32", h + 2)[0]
    for quant in ("f8", "i8", "mxfp8", "mxfp4"):
        whole = q.rmsnorm(x, w, res, quant=act(q, quant), y=True)
        for at in (slice(0, 300), slice(1099, 1100)):
            r = q.rmsnorm(x[at], w, None if res is None else res[at], quant=act(q, quant), y=True)
            for name, got, want in zip(r._fields, r, whole):
                if want is not None:
                    bits = [v.contiguous().view(torch.uint8) for v in (got, want[at])]
                    assert torch.equal(*bits), (name, quant, at)


@pytest.mark.parametrize("h", [512, 4096, 11008])
def test_the_sum_as_x(q, h):  # noqa: F811
    """The norm of x + residual, and of their sum given as x."""
    x, res = rows(1100, h, "f32", h), rows(1100, h, "f32", h + 1)
    w = rows(1, h, "f32", h + 2)[0]
    a = q.rmsnorm(x, w, res, quant=q.ACT_F8, y=True)
    b = q.rmsnorm(a.total, w, quant=q.ACT_F8, y=True)
    assert torch.equal(a.y, b.y) and torch.equal(a.scale, b.scale)


@pytest.mark.parametrize("n", [1, 300, 1100])
@pytest.mark.parametrize("weight", ["f32", "f16"])
@pytest.mark.parametrize("h", WIDTHS)
def test_near_the_formula(q, h, weight, n):  # noqa: F811
    x, w = rows(n, h, "f32", h + n), (1 + 0.3 * rows(1, h, "f32", 3)[0]).to(TYPES[weight])
    y = q.rmsnorm(x, w, eps=0.0, quant=None).y.double()
    t = x.double()
    ref = t / t.square().mean(1, keepdim=True).sqrt() * w.double()
    assert torch.all((y - ref).abs() <= 7 * U * ref.abs())


@pytest.mark.parametrize("h", [4096, 11008])
def test_near_the_formula_from_16_bits(q, h):  # noqa: F811
    """16-bit t and weights, seen through the scales of int8 codes (fp32: y's largest, over 127)."""
    for dtype in ("bf16", "f16"):
        x, w = rows(300, h, dtype, h), rows(1, h, dtype, h + 1)[0]
        got = q.rmsnorm(x, w, eps=0.0, quant=q.ACT_I8).scale.double()
        t = x.double()
        ref = (t / t.square().mean(1, keepdim=True).sqrt() * w.double()).abs().amax(1) / 127
        assert torch.all((got - ref).abs() <= 7 * U * ref)  # 6 u, and the division


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("name", ["mxfp4", "mxfp8"])
def test_on_borders_and_beside_them(q, name, dtype):  # noqa: F811
    """x of +-2: y is +-weight, exactly on the middle of two codes, on a power of two, or an ulp
    beside it; zeros and rows of blocks of zeros too.  The quantizer's own bytes."""
    rng = np.random.default_rng(1)
    h = 8192
    table = np.array(E2M1 if name == "mxfp4" else E4M3)
    points = np.concatenate([(table[1:] + table[:-1]) / 2, table, [table[-1] * 1.125]]).astype(np.float32)
    w = rng.choice(points, (h // 32, 32))
    w = np.where(rng.random(w.shape) < 0.6, np.nextafter(w, np.float32(rng.choice([-1e30, 1e30], w.shape))), w).astype(np.float32)
    w *= 2.0 ** rng.integers(-40, 40, (h // 32, 1))
    w[5::16] = 0
    w = torch.from_numpy(w.astype(np.float32).reshape(-1)).cuda()
    sign = torch.from_numpy(rng.choice([-1.0, 1.0], (40, h)).astype(np.float32)).cuda()
    r = q.rmsnorm((2 * sign).to(TYPES[dtype]), w, eps=0.0, quant=act(q, name))
    codes, scale = getattr(q, f"quantize_{name}")(sign * w)
    assert torch.equal(r.scale.view(torch.uint8), scale.view(torch.uint8))
    assert torch.equal(r.codes.view(torch.uint8), codes.view(torch.uint8))
