"""Timed cases of the operators around microscaled products: OCP microscaling
(MX) with 32 neighbouring values under one power-of-two scale, weights in 4 bits
(e2m1), activations in 4 or 8 (e4m3), and the norm that such activations come from.

    norm         t = x + residual, y = t / sqrt(mean(t^2) + eps) * weight, and y in 8
                 bits with scales: e4m3 with an fp32 scale per 128 columns, or MX
    quantize     a matrix to 4-bit MX codes and scales, and the values they stand for
    linear       y = W x, W in 4-bit MX, x quantized to MX in the call
    norm_linear  the norm with MX codes as its output, and the product of those codes:
                 what a decoder does before its attention and its feed-forward layer

Every case is synthetic: seeded normal activations with some large channels,
normal weights whose rows differ in spread.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BLOCK = 32  # values under one MX scale
GROUP = 128  # columns under one fp32 scale of the 8-bit format
TOP = {"mxfp4": (2, 6.0), "mxfp8": (8, 448.0)}  # exponent of the largest element, and its value
EPS = 1e-6


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one decoded token before a layer with 8-bit weights: the smallest call
        dict(name="norm-1", op="norm", n=1, h=4096, quant="f8", residual=True, dtype="bf16"),
        # a short prompt in wide rows, no residual (the first norm of a model)
        dict(name="norm-333", op="norm", n=333, h=11008, quant="mxfp8", residual=False, dtype="f16"),
        # a long prompt
        dict(name="norm-4096", op="norm", n=4096, h=4096, quant="f8", residual=True, dtype="bf16"),
        # a square projection of a 16-bit checkpoint converted, and looked at
        dict(name="quantize-4096", op="quantize", m=4096, k=4096, dtype="bf16"),
        # a large matrix of an fp32 checkpoint, ragged rows
        dict(name="quantize-5003", op="quantize", m=5003, k=11008, dtype="f32"),
        # one decoded token through a square projection
        dict(name="linear-1", op="linear", n=1, m=4096, k=4096, act="mxfp8", dtype="bf16"),
        # a few sequences decoded together, gate/up-like
        dict(name="linear-13", op="linear", n=13, m=11008, k=4096, act="mxfp4", dtype="f16"),
        # a larger decode batch, down-like
        dict(name="linear-64", op="linear", n=64, m=4096, k=14336, act="mxfp8", dtype="bf16"),
        # a short prompt through a matrix whose rows fill no whole tile (a vocabulary slice), fp32 results
        dict(name="linear-333", op="linear", n=333, m=5003, k=11008, act="mxfp4", dtype="f32"),
        # a long prompt: the largest product
        dict(name="linear-4096", op="linear", n=4096, m=14336, k=4096, act="mxfp4", dtype="bf16"),
        # one decoded token: norm, then gate and up of a 7B-shaped layer
        dict(name="norm-linear-1", op="norm_linear", n=1, m=22016, k=4096, act="mxfp8", dtype="bf16"),
        # the same for a prompt of odd length
        dict(name="norm-linear-1501", op="norm_linear", n=1501, m=22016, k=4096, act="mxfp8", dtype="f16"),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _near(rng, lo, hi, step):
    """A multiple of step in [lo, hi], spread over the logarithm."""
    return max(lo, min(hi, round(_spread(rng, lo, hi) / step) * step))


def draw(rng):
    op = rng.choice(["norm", "quantize", "linear", "norm_linear"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op == "norm":
        quant = rng.choice(["f8", "mxfp8"])
        h = _near(rng, 512, 11008, GROUP if quant == "f8" else BLOCK)
        n = min(4096 * 4096 // h, _spread(rng, 1, 4096))
        return dict(op=op, n=n, h=h, quant=quant, residual=rng.random() < 0.7, dtype=dtype)
    if op == "quantize":
        k = _near(rng, 256, 14336, BLOCK)
        return dict(op=op, m=min(5003 * 11008 // k, _spread(rng, 64, 14336)), k=k, dtype=dtype)
    if op == "norm_linear" and dtype == "f32":
        dtype = "bf16"  # a code next to a border moves an fp32 result by more than the sums' own rounding
    act, m, k = rng.choice(["mxfp4", "mxfp8"]), _spread(rng, 300, 22016), _near(rng, 512, 14336, BLOCK)
    most = 4096 * 14336 * 4096 // (m * k) // 2  # no more work than the largest listed product
    n = _spread(rng, 1, 4096 if op == "linear" else 1501)
    return dict(op=op, n=min(n, most), m=m, k=k, act=act, dtype=dtype)


def work(case):
    c, io = case, 4 if case["dtype"] == "f32" else 2
    if c["op"] == "norm":
        n, h = c["n"], c["h"]
        scales = n * h // GROUP * 4 if c["quant"] == "f8" else n * h // BLOCK
        return dict(bytes=n * h * (io * (3 if c["residual"] else 1) + 1) + scales + h * io, flops=n * h * 8)
    m, k = c["m"], c["k"]
    if c["op"] == "quantize":
        return dict(bytes=m * k * 2 * io + m * k // BLOCK, flops=m * k * 4)
    n = c["n"]
    weights = m * k // 2 + m * k // BLOCK
    if c["op"] == "linear":
        return dict(bytes=weights + n * (k + m) * io, flops=2 * n * m * k)
    return dict(bytes=weights + n * (3 * k + m) * io + k * io, flops=2 * n * m * k)


# ----------------------------------------------------------------- the inputs
def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _activations(g, n, k, dtype):
    x = torch.randn(n, k, generator=g, device="cuda")
    loud = torch.rand(k, generator=g, device="cuda") < 0.01  # a few channels an order of magnitude above the rest
    return torch.where(loud, x * 10.0, x).to(DTYPES[dtype])


def _matrix(g, m, k):
    w = torch.randn(m, k, generator=g, device="cuda")
    return w * (0.02 * torch.exp(torch.rand(m, 1, generator=g, device="cuda") * 2.0 - 1.0))


def _inputs(case, seed):
    c, g = case, _generator(seed)
    if c["op"] == "quantize":
        return dict(w=_matrix(g, c["m"], c["k"]).to(DTYPES[c["dtype"]]))
    s = {}
    if c["op"] != "linear":
        n, h = c["n"], c["h"] if c["op"] == "norm" else c["k"]
        s["weight"] = (1.0 + 0.1 * torch.randn(h, generator=g, device="cuda")).to(DTYPES[c["dtype"]])
        s["residual"] = _activations(g, n, h, c["dtype"]) if c.get("residual", True) else None
        s["x"] = torch.randn(n, h, generator=g, device="cuda").to(DTYPES[c["dtype"]])
    else:
        s["x"] = _activations(g, c["n"], c["k"], c["dtype"])
    if c["op"] != "norm":
        q, e = _plain_mx(_matrix(g, c["m"], c["k"]), "mxfp4")
        s["wq"], s["ws"] = _pack(q), (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)
    return s


def prepare(case, seed):
    return dict(case) | _inputs(case, seed)


# ------------------------------------------------------------------ one pass
def run(state):
    s = state
    if own:
        import bit_block_quant_amd as qblk

        if s["op"] == "norm":
            r = qblk.rmsnorm(s["x"], s["weight"], residual=s["residual"], eps=EPS, quant=qblk.ACTS[s["quant"]])
            return dict(codes=r.codes, scale=r.scale, total=r.total)
        if s["op"] == "quantize":
            codes, scale = qblk.quantize_mxfp4(s["w"])
            return dict(values=qblk.dequant_mx(codes, scale, s["w"].dtype), scale=scale)
        if s["op"] == "linear":
            return qblk.linear_mxfp4(s["x"], s["wq"], s["ws"], act=qblk.ACTS[s["act"]])
        r = qblk.rmsnorm(s["x"], s["weight"], residual=s["residual"], eps=EPS, quant=qblk.ACTS[s["act"]])
        return dict(y=qblk.gemm_mxfp4(s["wq"], s["ws"], r.codes, r.scale, dtype=s["x"].dtype), total=r.total)
    if s["op"] == "norm":
        y, total = _plain_norm(s)
        if s["quant"] == "f8":
            codes, scale = _plain_f8(y)
        else:
            q, e = _plain_mx(y, s["quant"])
            codes, scale = q.to(torch.float8_e4m3fn), (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)
        return dict(codes=codes, scale=scale, total=total)
    if s["op"] == "quantize":
        q, e = _plain_mx(s["w"].float(), "mxfp4")
        return dict(values=_plain_values(q, e).to(s["w"].dtype), scale=(e + 127).to(torch.uint8).view(torch.float8_e8m0fnu))
    y, total = (s["x"].float(), None) if s["op"] == "linear" else _plain_norm(s)
    x = _plain_values(*_plain_mx(y, s["act"]))
    y = (x @ _plain_weights(s["wq"], s["ws"]).t()).to(s["x"].dtype)
    return y if s["op"] == "linear" else dict(y=y, total=total)


def _plain_norm(s):
    """The normalized values in fp32, and the sum that is normalized, of x's type (None without a residual)."""
    total = None if s["residual"] is None else (s["x"].float() + s["residual"].float()).to(s["x"].dtype)
    t = (s["x"] if total is None else total).float()
    return t / torch.sqrt((t * t).mean(-1, keepdim=True) + EPS) * s["weight"].float(), total


def _plain_f8(y):
    t = y.view(y.shape[0], -1, GROUP)
    # a tensor on the device as divisor: both quotients are rounded once (a Python number would be multiplied by its reciprocal)
    scale = t.abs().amax(-1, keepdim=True) / torch.full((), 448.0, device=y.device)
    codes = torch.where(scale == 0, 0.0, t / scale).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return codes.view_as(y), scale[..., 0]


def _plain_mx(v, elem):
    """fp32 values (rows, k) -> the elements as fp32 (rows, k), and the exponents of the scales (rows, k/32)."""
    top, most = TOP[elem]
    t = v.view(v.shape[0], -1, BLOCK)
    big = t.abs().amax(-1)
    _, e = torch.frexp(big)  # big = f * 2^e, f in [0.5, 1)
    e = torch.where(big == 0, -127, (e - 1 - top).clamp(-127, 127))
    q = (t * torch.exp2(-e.double()).float()[..., None]).clamp(-most, most)
    if elem == "mxfp8":
        q = q.to(torch.float8_e4m3fn).float()
    else:  # steps of 1/2 below 2, 1 below 4, 2 below 6; torch rounds halves to even, as the format does
        step = torch.where(q.abs() < 2, 0.5, torch.where(q.abs() < 4, 1.0, 2.0))
        q = torch.round(q / step) * step
    return q.view_as(v), e


def _plain_values(q, e):
    return (q.view(q.shape[0], -1, BLOCK) * torch.exp2(e.double()).float()[..., None]).view_as(q)


def _pack(q):
    """e2m1 values (rows, k) -> their codes, two to a byte, the even column's in the low half."""
    a = q.abs()
    code = torch.where(a < 2, a * 2, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)  # 0 .5 1 1.5 2 3 4 6 -> 0..7
    code = code + 8 * torch.signbit(q).to(torch.uint8)
    return code[:, ::2] | (code[:, 1::2] << 4)


def _plain_weights(wq, ws):
    code = torch.stack([wq & 15, wq >> 4], -1).flatten(-2)
    c = (code & 7).float()
    a = torch.where(c < 4, c / 2, torch.where(c < 6, c - 2, c * 2 - 8))
    q = torch.where(code >= 8, -a, a)
    return (q.view(q.shape[0], -1, BLOCK) * ws.float()[..., None]).view_as(q)


# ------------------------------------------------------------- in 64 bits
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _power(e):
    """2^e in 64 bits for whole e in [-300, 300], looked up: the device's power function is not exact there."""
    return torch.tensor([2.0 ** i for i in range(-300, 301)], dtype=torch.float64, device=e.device)[e.long() + 300]


def _exact_mx(v, elem):
    """float64 values (rows, k) -> their MX elements and scales in 64 bits, by comparison with the formats' values."""
    if elem == "mxfp4":
        table = E2M1
    else:
        table = [m * 2.0 ** -9 for m in range(8)] + [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)][:-1]
    values = torch.tensor(table, dtype=torch.float64, device=v.device)
    t = v.view(v.shape[0], -1, BLOCK)
    big = t.abs().max(dim=-1).values
    safe = torch.where(big > 0, big, 1.0)
    e = torch.floor(torch.log2(safe))
    e = e + (_power(e + 1) <= safe).double() - (_power(e) > safe).double()  # next to a power of two the logarithm may be rounded past it
    e = torch.where(big > 0, e - math.floor(math.log2(table[-1])), -127.0).clamp(-127, 127)
    scale = _power(e)
    a = (t / scale[..., None]).abs()
    at = torch.searchsorted(values, a).clamp(1, len(table) - 1)  # values[at - 1] < a <= values[at], or the last pair
    down, up = a - values[at - 1], values[at] - a
    index = torch.where((up < down) | ((up == down) & (at % 2 == 0)), at, at - 1)
    return torch.copysign(values[index], t).view_as(v), scale


def _exact_norm(case, s):
    total = None if s["residual"] is None else (s["x"].double() + s["residual"].double()).to(DTYPES[case["dtype"]])
    t = (s["x"] if total is None else total).double()
    rms = (t.square().sum(dim=1, keepdim=True) / t.shape[1] + EPS).sqrt()
    return t / rms * s["weight"].double(), None if total is None else total.double()


def _exact_product(x, wq, ws):
    table = torch.tensor(E2M1 + [-v for v in E2M1], dtype=torch.float64, device=x.device)
    y = torch.empty(x.shape[0], wq.shape[0], dtype=torch.float64, device=x.device)
    for r in range(0, wq.shape[0], 1024):
        b = wq[r:r + 1024].long()
        w = torch.empty(b.shape[0], 2 * b.shape[1], dtype=torch.float64, device=x.device)
        w[:, 0::2], w[:, 1::2] = table[b % 16], table[b // 16]
        y[:, r:r + 1024] = x @ (w * ws[r:r + 1024].double().repeat_interleave(BLOCK, 1)).t()
    return y


def exact(case, seed):
    c, s = case, _inputs(case, seed)
    if c["op"] == "norm":
        y, total = _exact_norm(c, s)
        if c["quant"] == "mxfp8":
            codes, scale = _exact_mx(y, "mxfp8")
            return dict(codes=codes, scale=scale, total=total)
        g = y.view(y.shape[0], -1, GROUP)
        scale = g.abs().max(dim=-1).values / 448.0
        a = g / torch.where(scale > 0, scale, 1.0)[..., None]
        _, e = torch.frexp(a)
        step = _power((e - 1).clamp(min=-6) - 3)
        return dict(codes=(torch.round(a / step) * step).view_as(y), scale=scale, total=total)
    if c["op"] == "quantize":
        q, scale = _exact_mx(s["w"].double(), "mxfp4")
        return dict(values=q * scale.repeat_interleave(BLOCK, 1), scale=scale)
    y, total = (s["x"].double(), None) if c["op"] == "linear" else _exact_norm(c, s)
    q, scale = _exact_mx(y, c["act"])
    y = _exact_product(q * scale.repeat_interleave(BLOCK, 1), s["wq"], s["ws"])
    return y if c["op"] == "linear" else dict(y=y, total=total)
