"""Timed cases of the feed-forward operators: 8-bit floating point products with
a scale for each block of 128, the gated feed-forward layer built from them, and
a whole mixture-of-experts layer whose experts are packed 4-bit matrices.

    linear_f8   y = W x: x is quantized to e4m3 per token and 128 columns, W is
                e4m3 with one fp32 scale per 128 x 128 weights
    ffn_f8      y = W2 (silu(Wg x) * (Wu x)), all three matrices as above, the
                product of the two halves quantized like x
    moe         y = sum over a token's top_k experts of w_e * D_e (silu(G_e x) *
                (U_e x)), the experts chosen from given router logits

Every case is synthetic: seeded normal activations with some large channels,
normal weights whose rows (or experts) differ in spread.
"""
import math

import torch

own = False

F8_MAX = 448.0  # largest finite e4m3 value
GROUP = 128
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
# weights and bytes of one block of each packed 4-bit format
BLOCK = {"q4_0": (32, 18), "sb4": (256, 138), "sb4_affine": (256, 148), "q4_k": (256, 144)}


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one decoded token through a square projection: the smallest call
        dict(name="linear-1", op="linear_f8", n=1, m=4096, k=4096, dtype="bf16"),
        # a few sequences decoded together, gate/up-like
        dict(name="linear-13", op="linear_f8", n=13, m=11008, k=4096, dtype="f16"),
        # a short prompt through a matrix whose rows fill no whole block (a vocabulary slice)
        dict(name="linear-333", op="linear_f8", n=333, m=5003, k=11008, dtype="bf16"),
        # a long prompt: the largest product
        dict(name="linear-4096", op="linear_f8", n=4096, m=14336, k=4096, dtype="bf16"),
        # the dense layer of a 7B-shaped model, one token
        dict(name="ffn-1", op="ffn_f8", n=1, h=4096, i=11008, dtype="bf16"),
        # an 8B-shaped layer, a decode batch
        dict(name="ffn-32", op="ffn_f8", n=32, h=4096, i=14336, dtype="f16"),
        # a prompt of odd length
        dict(name="ffn-1501", op="ffn_f8", n=1501, h=4096, i=11008, dtype="bf16"),
        # many small experts, one token: latency counts
        dict(name="moe-1", op="moe", n=1, e=64, top_k=8, h=2048, i=1024, fmt="sb4", dtype="f16", renorm=True, masked=False),
        # few large experts, one token
        dict(name="moe-1-large", op="moe", n=1, e=8, top_k=2, h=4096, i=14336, fmt="q4_k", dtype="bf16", renorm=True, masked=False),
        # a decode batch that reaches most of the small experts
        dict(name="moe-16", op="moe", n=16, e=64, top_k=8, h=2048, i=1024, fmt="q4_0", dtype="bf16", renorm=False, masked=False),
        # an odd batch with unused slots (no expert left) and experts switched off
        dict(name="moe-29-masked", op="moe", n=29, e=128, top_k=8, h=4096, i=1280, fmt="sb4", dtype="f16", renorm=True, masked=True),
        # the largest batch the layer is meant for
        dict(name="moe-64", op="moe", n=64, e=32, top_k=4, h=4096, i=2048, fmt="sb4_affine", dtype="bf16", renorm=True, masked=False),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _near(rng, lo, hi, step):
    """A multiple of step in [lo, hi], spread over the logarithm; 3072 is moved one step up."""
    v = max(lo, min(hi, round(_spread(rng, lo, hi) / step) * step))
    return v + step if v == 3072 else v


def draw(rng):
    op = rng.choice(["linear_f8", "ffn_f8", "moe"])
    dtype = rng.choice(["bf16", "f16"])
    if op == "linear_f8":
        m = _spread(rng, 300, 14336)
        k = _near(rng, 512, 11008, 128)
        most = 4096 * 14336 * 4096 // (m * k)  # no more work than the largest listed product
        return dict(op=op, n=min(most, _spread(rng, 1, 4096)), m=m + (m == 3072), k=k, dtype=dtype)
    if op == "ffn_f8":
        return dict(op=op, n=_spread(rng, 1, 1501), h=_near(rng, 512, 4096, 128), i=_near(rng, 512, 11008, 128), dtype=dtype)
    fmt = rng.choice(sorted(BLOCK))
    step = 32 if fmt == "q4_0" else 256
    e, top_k = rng.choice([(8, 2), (16, 2), (32, 4), (64, 6), (64, 8), (128, 8)])
    i = _near(rng, 256, 8192 if e <= 16 else 1280, step)
    return dict(op=op, n=_spread(rng, 1, 64), e=e, top_k=top_k, h=_near(rng, 512, 4096, step), i=i + step * (2 * i == 3072),
                fmt=fmt, dtype=dtype, renorm=rng.random() < 0.5, masked=rng.random() < 0.3)


def work(case):
    c, io = case, 2
    if c["op"] == "linear_f8":
        n, m, k = c["n"], c["m"], c["k"]
        return dict(bytes=_f8_bytes(m, k) + n * (k + m) * io, flops=2 * n * m * k)
    n, h, i = c["n"], c["h"], c["i"]
    if c["op"] == "ffn_f8":
        return dict(bytes=_f8_bytes(2 * i, h) + _f8_bytes(h, i) + 2 * n * h * io, flops=6 * n * h * i)
    # experts that at least one token takes, where every expert is as likely (of the
    # masked cases, three tokens in four are in use and three experts in four are on)
    live_n, live_e = (n - n // 4, c["e"] - c["e"] // 4) if c["masked"] else (n, c["e"])
    reached = live_e * (1.0 - (1.0 - min(1.0, c["top_k"] / live_e)) ** live_n)
    weights, size = BLOCK[c["fmt"]]
    return dict(bytes=int(reached * 3 * h * i / weights * size) + 2 * n * h * io + n * c["e"] * 4 + n * c["top_k"] * 8,
                flops=6 * live_n * c["top_k"] * h * i)


def _f8_bytes(rows, k):
    return rows * k + 4 * (-(-rows // GROUP)) * (k // GROUP)


# ----------------------------------------------------------------- the inputs
def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _activations(g, n, k, dtype):
    x = torch.randn(n, k, generator=g, device="cuda")
    loud = torch.rand(k, generator=g, device="cuda") < 0.01  # a few channels an order of magnitude above the rest
    return torch.where(loud, x * 10.0, x).to(DTYPES[dtype])


def _f8_weights(g, rows, k, std):
    """e4m3 codes (rows, k) and fp32 scales (ceil(rows/128), k/128) of a normal matrix."""
    w = torch.randn(rows, k, generator=g, device="cuda")
    w *= std * torch.exp(torch.rand(rows, 1, generator=g, device="cuda") * 2.0 - 1.0)
    blocks = -(-rows // GROUP)
    padded = torch.zeros(blocks * GROUP, k, device="cuda")
    padded[:rows] = w
    tiles = padded.view(blocks, GROUP, k // GROUP, GROUP)
    scale = tiles.abs().amax(dim=(1, 3)) / F8_MAX
    codes = (tiles / scale[:, None, :, None]).clamp(-F8_MAX, F8_MAX).view(blocks * GROUP, k)[:rows]
    return codes.to(torch.float8_e4m3fn).contiguous(), scale.contiguous()


def _half_bytes(v):
    return v.to(torch.float16).contiguous().view(torch.uint8).view(*v.shape, 2)


def _nibbles(codes):
    """(..., 32) codes 0..15 -> (..., 16) bytes: code j low, code j+16 high."""
    c = codes.to(torch.uint8)
    return c[..., :16] | (c[..., 16:] << 4)


def _pack(g, fmt, rows, k, std):
    """A normal matrix as packed 4-bit blocks (uint8, rows * k / E * B bytes)."""
    elems, size = BLOCK[fmt]
    w = torch.randn(rows, k // elems, elems // 32, 32, generator=g, device="cuda")
    w *= std
    out = torch.empty(rows, k // elems, size, dtype=torch.uint8, device="cuda")
    lo, hi = w.amin(-1), w.amax(-1)  # per 32 weights: (rows, k/E, E/32)
    if fmt in ("q4_0", "sb4"):
        d = (torch.maximum(hi, -lo) / 7.0).half().float()
        q = _nibbles((w / d[..., None]).round().clamp(-8, 7) + 8)
        if fmt == "q4_0":
            out[..., :2] = _half_bytes(d[..., 0])
            out[..., 2:] = q[..., 0, :]
        else:
            top = (d.amax(-1) / 127.0).half().float()
            out[..., :2] = _half_bytes(top)
            out[..., 2:10] = (d / top[..., None]).round().clamp(-127, 127).to(torch.int8).view(torch.uint8)
            out[..., 10:] = q.flatten(-2)
    elif fmt == "sb4_affine":
        d = ((hi - lo) / 15.0).half().float()
        a = lo.half().float()
        q = _nibbles(((w - a[..., None]) / d[..., None]).round().clamp(0, 15))
        for at, v in ((0, d), (1, a)):
            top = (v.abs().amax(-1) / 127.0).half().float()
            out[..., 2 * at:2 * at + 2] = _half_bytes(top)
            out[..., 4 + 8 * at:12 + 8 * at] = (v / top[..., None]).round().clamp(-127, 127).to(torch.int8).view(torch.uint8)
        out[..., 20:] = q.flatten(-2)
    else:
        lo = lo.clamp(max=0.0)
        d, dmin = ((hi - lo) / 15.0), -lo
        fields = torch.zeros(*d.shape[:-1], 16, dtype=torch.int64, device="cuda")
        for at, v in ((0, d), (1, dmin)):
            top = (v.amax(-1) / 63.0).half().float()
            out[..., 2 * at:2 * at + 2] = _half_bytes(top)
            fields[..., 8 * at:8 * at + 8] = (v / top[..., None]).round().clamp(0, 63).to(torch.int64)
        # sixteen 6-bit fields, four to three bytes
        f = fields.view(*d.shape[:-1], 4, 4)
        word = f[..., 0] | (f[..., 1] << 6) | (f[..., 2] << 12) | (f[..., 3] << 18)
        out[..., 4:16] = torch.stack([word & 255, (word >> 8) & 255, word >> 16], -1).flatten(-2).to(torch.uint8)
        q = _nibbles(((w - lo[..., None]) / d[..., None]).round().clamp(0, 15))
        out[..., 16:] = q.flatten(-2)
    return out.view(-1)


def _inputs(case, seed):
    c, g = case, _generator(seed)
    x = _activations(g, c["n"], c["k"] if c["op"] == "linear_f8" else c["h"], c["dtype"])
    if c["op"] == "linear_f8":
        wq, ws = _f8_weights(g, c["m"], c["k"], 0.02)
        return dict(x=x, wq=wq, ws=ws)
    if c["op"] == "ffn_f8":
        w13, s13 = _f8_weights(g, 2 * c["i"], c["h"], 0.02)
        w2, s2 = _f8_weights(g, c["h"], c["i"], 0.02)
        return dict(x=x, w13=w13, s13=s13, w2=w2, s2=s2)
    n, e = c["n"], c["e"]
    logits = torch.randn(n, e, generator=g, device="cuda") * 1.5
    if c["masked"]:
        off = torch.rand(e, generator=g, device="cuda").argsort()[: e // 4]  # experts switched off
        logits[:, off] = -torch.inf
        idle = torch.rand(n, generator=g, device="cuda").argsort()[: n // 4]  # unused slots of the batch
        logits[idle] = -torch.inf
    return dict(x=x, logits=logits, gate_up=_pack(g, c["fmt"], e * 2 * c["i"], c["h"], 0.02),
                down=_pack(g, c["fmt"], e * c["h"], c["i"], 0.02))


def prepare(case, seed):
    return dict(case) | _inputs(case, seed)


# ------------------------------------------------------------------ one pass
def run(state):
    s = state
    if own:
        import bit_block_quant_amd as qblk

        if s["op"] == "linear_f8":
            return qblk.linear_f8(s["x"], s["wq"], s["ws"])
        if s["op"] == "ffn_f8":
            return qblk.ffn_f8(s["x"], s["w13"], s["s13"], s["w2"], s["s2"])
        y, ids, weights = qblk.moe(qblk.FORMATS[s["fmt"]], s["x"], s["logits"], s["gate_up"], s["down"], s["i"],
                                   s["top_k"], renorm=s["renorm"])
        return dict(y=y, ids=ids, weights=weights)
    if s["op"] == "linear_f8":
        return (_plain_act(s["x"].float()) @ _plain_weights(s["wq"], s["ws"]).t()).to(s["x"].dtype)
    if s["op"] == "ffn_f8":
        gu = _plain_act(s["x"].float()) @ _plain_weights(s["w13"], s["s13"]).t()
        y = _plain_act(_plain_gate(gu)) @ _plain_weights(s["w2"], s["s2"]).t()
        return y.to(s["x"].dtype)
    return _plain_moe(s)


def _plain_act(x):
    """x quantized to e4m3 per row and 128 columns, as the values the codes stand for."""
    t = x.view(x.shape[0], -1, GROUP)
    # a tensor on the device as divisor: both quotients are rounded once (a Python number would be multiplied by its reciprocal)
    scale = t.abs().amax(-1, keepdim=True) / torch.full((), F8_MAX, device=x.device)
    codes = torch.where(scale == 0, 0.0, t / scale).clamp(-F8_MAX, F8_MAX).to(torch.float8_e4m3fn)
    return (codes.float() * scale).view_as(x)


def _plain_weights(wq, ws):
    rows, k = wq.shape
    spread = ws.repeat_interleave(GROUP, 0)[:rows]
    return (wq.float().view(rows, -1, GROUP) * spread[..., None]).view(rows, k)


def _plain_gate(gu):
    gate, up = gu.chunk(2, -1)
    return gate / (1.0 + torch.exp(-gate)) * up


def _plain_unpack(blocks, fmt):
    """Packed blocks (..., B bytes) -> their weights (..., E) in fp32."""
    def half(at):
        return blocks[..., at:at + 2].contiguous().view(torch.float16).float()

    def bytes8(at):
        return blocks[..., at:at + 8].contiguous().view(torch.int8).float()

    at = {"q4_0": 2, "sb4": 10, "sb4_affine": 20, "q4_k": 16}[fmt]
    qs = blocks[..., at:].unflatten(-1, (-1, 16))
    codes = torch.cat([qs & 15, qs >> 4], -1).float()  # (..., E/32, 32)
    if fmt == "q4_0":
        w = half(0)[..., None] * (codes - 8.0)
    elif fmt == "sb4":
        w = (half(0) * bytes8(2))[..., None] * (codes - 8.0)
    elif fmt == "sb4_affine":
        w = (half(0) * bytes8(4))[..., None] * codes + (half(2) * bytes8(12))[..., None]
    else:
        b = blocks[..., 4:16].unflatten(-1, (4, 3)).int()
        word = b[..., 0] | (b[..., 1] << 8) | (b[..., 2] << 16)
        fields = torch.stack([word & 63, (word >> 6) & 63, (word >> 12) & 63, word >> 18], -1).flatten(-2).float()
        w = (half(0) * fields[..., :8])[..., None] * codes - (half(2) * fields[..., 8:])[..., None]
    return w.flatten(-2)


def _plain_route(logits, top_k, renorm):
    """ids (n, top_k) int32, -1 where no expert is left, and weights (n, top_k)."""
    value, index = torch.sort(logits, dim=-1, descending=True, stable=True)  # equal logits: the lowest index first
    on = value > -torch.inf
    p = torch.where(on, torch.exp(value - torch.where(on[:, :1], value[:, :1], 0.0)), 0.0)
    total = (p[:, :top_k] if renorm else p).sum(-1, keepdim=True)
    weights = torch.where(on[:, :top_k], p[:, :top_k] / total, 0.0)
    return torch.where(on[:, :top_k], index[:, :top_k], -1).int(), weights


def _plain_moe(s):
    n, e, h, i, top_k, fmt = s["x"].shape[0], s["e"], s["h"], s["i"], s["top_k"], s["fmt"]
    elems, size = BLOCK[fmt]
    x = s["x"].float()
    ids, weights = _plain_route(s["logits"], top_k, s["renorm"])
    at = ids.clamp(min=0).long()
    gate_up, down = s["gate_up"].view(e, 2 * i, h // elems, size), s["down"].view(e, h, i // elems, size)
    if n * top_k <= e:
        # few pairs of token and expert: each with its own expert's matrices
        pairs = at.flatten()
        gu = torch.bmm(_plain_unpack(gate_up[pairs], fmt).flatten(2), x.repeat_interleave(top_k, 0)[:, :, None])[..., 0]
        y = torch.bmm(_plain_unpack(down[pairs], fmt).flatten(2), _plain_gate(gu)[:, :, None])[..., 0]
        y = (y.view(n, top_k, h) * weights[..., None]).sum(1)
    else:
        # every expert for every token, the ones not taken at weight zero
        dense = torch.zeros(n, e, device=x.device).scatter_add_(1, at, weights)
        gu = (x @ _plain_unpack(gate_up, fmt).view(e * 2 * i, h).t()).view(n, e, 2 * i)
        mid = (_plain_gate(gu) * dense[..., None]).transpose(0, 1)
        y = torch.bmm(mid.contiguous(), _plain_unpack(down, fmt).view(e, h, i).transpose(1, 2).contiguous()).sum(0)
    return dict(y=y.to(s["x"].dtype), ids=ids, weights=weights)


# ------------------------------------------------------------- in 64 bits
def _round_e4m3(v):
    """float64 values in [-448, 448] to the nearest e4m3 value, ties to even."""
    _, exponent = torch.frexp(v)  # v = f * 2^exponent, f in [0.5, 1)
    step = torch.ldexp(torch.ones_like(v), (exponent - 1).clamp(min=-6) - 3)
    return torch.round(v / step) * step


def _exact_act(x):
    """The quantized x in 64 bits.  By definition the scale and the quotient that
    is rounded to e4m3 are fp32 numbers: 16-bit inputs often meet a tie exactly."""
    out = torch.empty_like(x)
    for c in range(0, x.shape[1], GROUP):
        t = x[:, c:c + GROUP]
        scale = (t.abs().max(dim=1, keepdim=True).values / 448.0).float().double()
        safe = torch.where(scale > 0, scale, 1.0)
        out[:, c:c + GROUP] = _round_e4m3((t / safe).float().double().clamp(-448.0, 448.0)) * scale
    return out


def _exact_product(x, wq, ws):
    y = torch.empty(x.shape[0], wq.shape[0], dtype=torch.float64, device=x.device)
    for r in range(0, wq.shape[0], GROUP):
        w = wq[r:r + GROUP].to(torch.float64)
        y[:, r:r + GROUP] = x @ (w * ws[r // GROUP].double().repeat_interleave(GROUP)).t()
    return y


def _exact_matrix(raw, fmt, rows, k):
    """One packed matrix (uint8, flat) in 64 bits."""
    elems, size = BLOCK[fmt]
    b = raw.view(rows * k // elems, size).long()

    def f16(lo):
        return (b[:, lo] | (b[:, lo + 1] << 8)).to(torch.int16).view(torch.float16).double()

    def i8(j):
        return ((b[:, j] ^ 128) - 128).double()

    w = torch.empty(b.shape[0], elems, dtype=torch.float64, device=raw.device)
    start = size - elems // 2
    bits = [sum(b[:, 4 + j + 3 * t] << (8 * j) for j in range(3)) for t in range(4)] if fmt == "q4_k" else None
    for u in range(elems // 32):
        if fmt == "q4_0":
            scale, shift = f16(0), -8.0 * f16(0)
        elif fmt == "sb4":
            scale = f16(0) * i8(2 + u)
            shift = -8.0 * scale
        elif fmt == "sb4_affine":
            scale, shift = f16(0) * i8(4 + u), f16(2) * i8(12 + u)
        else:
            scale = f16(0) * ((bits[u // 4] >> (6 * (u % 4))) & 63).double()
            shift = -f16(2) * ((bits[2 + u // 4] >> (6 * (u % 4))) & 63).double()
        byte = b[:, start + 16 * u:start + 16 * u + 16]
        w[:, 32 * u:32 * u + 16] = scale[:, None] * (byte % 16) + shift[:, None]
        w[:, 32 * u + 16:32 * u + 32] = scale[:, None] * (byte // 16) + shift[:, None]
    return w.view(rows, k)


def exact(case, seed):
    c, s = case, _inputs(case, seed)
    x = s["x"].double()
    if c["op"] == "linear_f8":
        return _exact_product(_exact_act(x), s["wq"], s["ws"])
    if c["op"] == "ffn_f8":
        gu = _exact_product(_exact_act(x), s["w13"], s["s13"])
        gate = gu[:, :c["i"]]
        return _exact_product(_exact_act(gate * torch.sigmoid(gate) * gu[:, c["i"]:]), s["w2"], s["s2"])
    n, e, h, i, top_k = c["n"], c["e"], c["h"], c["i"], c["top_k"]
    ids, weights = [], []
    for row in s["logits"].double().cpu().tolist():
        order = [j for j in sorted(range(e), key=lambda j: (-row[j], j)) if row[j] > -math.inf]
        p = {j: math.exp(row[j] - row[order[0]]) for j in order}
        taken = order[:top_k]
        total = math.fsum(p[j] for j in (taken if c["renorm"] else order))
        ids.append(taken + [-1] * (top_k - len(taken)))
        weights.append([p[j] / total for j in taken] + [0.0] * (top_k - len(taken)))
    y = torch.zeros(n, h, dtype=torch.float64, device="cuda")
    up_bytes, down_bytes = s["gate_up"].numel() // e, s["down"].numel() // e
    for j in sorted({j for row in ids for j in row if j >= 0}):
        tokens = [t for t in range(n) if j in ids[t]]
        share = torch.tensor([weights[t][ids[t].index(j)] for t in tokens], dtype=torch.float64, device="cuda")
        gu = x[tokens] @ _exact_matrix(s["gate_up"][j * up_bytes:(j + 1) * up_bytes], c["fmt"], 2 * i, h).t()
        mid = gu[:, :i] * torch.sigmoid(gu[:, :i]) * gu[:, i:]
        d = _exact_matrix(s["down"][j * down_bytes:(j + 1) * down_bytes], c["fmt"], h, i)
        y[tokens] += share[:, None] * (mid @ d.t())
    return dict(y=y, ids=torch.tensor(ids, dtype=torch.int32, device="cuda"),
                weights=torch.tensor(weights, dtype=torch.float64, device="cuda"))
