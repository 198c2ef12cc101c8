"""The binding's refusals for the feed-forward operators (CPU only): every bad
argument raises before a compute entry point is reached."""
import pytest
import torch

from test_binding_checks import FakeGpuTensor, RecordingLib, pytestmark  # noqa: F401

F32, F16, BF16, U8, I32 = torch.float32, torch.float16, torch.bfloat16, torch.uint8, torch.int32
F8 = torch.float8_e4m3fn
M, K, N = 200, 256, 3


class Lib(RecordingLib):
    GEOMETRY = RecordingLib.GEOMETRY + ("qblk_gemm_f8_workspace", "qblk_linear_f8_workspace", "qblk_ffn_f8_workspace",
                                        "qblk_moe_workspace")


@pytest.fixture()
def q(monkeypatch):
    import bit_block_quant_amd as q
    rec = Lib(q._lib)
    monkeypatch.setattr(q, "_lib", rec)
    yield q
    assert rec.calls == [], f"a compute entry point was reached: {rec.calls}"


T = FakeGpuTensor
WQ, WS = T((M, K), F8), T((2, 2), F32)


def test_quantizers(q):
    with pytest.raises(ValueError, match="GPU tensor"):
        q.quantize_f8(torch.zeros(M, K))
    with pytest.raises(ValueError, match="multiple of 128"):
        q.quantize_f8(T((M, 200), F32), out=T((M, 200), F8), scale=T((2, 2), F32))
    with pytest.raises(ValueError, match="expected 4 elements"):
        q.quantize_f8(T((M, K), F32), out=WQ, scale=T((2, 1), F32))
    with pytest.raises(ValueError, match="expected 51200 elements"):
        q.quantize_f8(T((M, K), F32), out=T((M - 1, K), F8), scale=WS)
    with pytest.raises(TypeError, match="element type"):
        q.quantize_f8(T((M, K), F8), out=WQ, scale=WS)
    with pytest.raises(ValueError, match="contiguous"):
        q.quantize_act_f8(T((N, K), F16, contiguous=False))
    with pytest.raises(ValueError, match="multiple of 128"):
        q.quantize_act_f8(T((N, 64), F16))
    with pytest.raises(ValueError, match="scale: expected 6 elements"):
        q.quantize_act_f8(T((N, K), F16), out=T((N, K), F8), scale=T((N, 1), F32))
    with pytest.raises(TypeError, match="out: element type"):
        q.quantize_act_f8(T((N, K), F16), out=T((N, K), torch.int8), scale=T((N, 2), F32))


def test_products(q):
    x, y = T((N, K), BF16), T((N, M), BF16)
    with pytest.raises(ValueError, match="columns"):
        q.linear_f8(T((N, 128), BF16), WQ, WS, out=y)
    with pytest.raises(ValueError, match="scale: expected 4"):
        q.linear_f8(x, WQ, T((1, 2), F32), out=y)
    with pytest.raises(TypeError, match="element type"):
        q.linear_f8(x, T((M, K), BF16), WS, out=y)
    with pytest.raises(ValueError, match="expected 600 elements"):
        q.linear_f8(x, WQ, WS, out=T((N, M + 1), BF16))
    with pytest.raises(ValueError, match="other arguments"):
        q.linear_f8(T((N, K), BF16, index=1), WQ, WS, out=y)
    with pytest.raises(ValueError, match="workspace: holds"):
        q.linear_f8(T((70, K), BF16), WQ, WS, out=T((70, M), BF16), workspace=T((16,), U8))
    xq, xs = T((N, K), U8), T((N, 2), F32)
    with pytest.raises(ValueError, match="xs: expected 6"):
        q.gemm_f8(WQ, WS, xq, T((N,), F32), out=T((N, M), F32))
    with pytest.raises(TypeError, match="xq: element type"):
        q.gemm_f8(WQ, WS, T((N, K), F16), xs, out=T((N, M), F32))
    with pytest.raises(ValueError, match="dimensions"):
        q.gemm_f8(WQ, WS, T((N * K,), U8), xs, out=T((N, M), F32))


def test_gated_layer(q):
    w13, s13, w2, s2 = T((512, 128), F8), T((4, 1), F32), T((128, 256), F8), T((1, 2), F32)
    x, y = T((N, 128), F16), T((N, 128), F16)
    work = T((1 << 20,), U8)
    with pytest.raises(ValueError, match="gated layer"):
        q.ffn_f8(x, T((256, 128), F8), T((2, 1), F32), w2, s2, out=y, workspace=work)
    with pytest.raises(ValueError, match="gated layer"):
        q.ffn_f8(T((N, 256), F16), T((512, 256), F8), T((4, 2), F32), w2, s2, out=y, workspace=work)
    with pytest.raises(ValueError, match="w2 scale"):
        q.ffn_f8(x, w13, s13, w2, T((2, 2), F32), out=y, workspace=work)
    with pytest.raises(ValueError, match="x: expected 128 columns"):
        q.ffn_f8(T((N, 256), F16), w13, s13, w2, s2, out=y, workspace=work)
    with pytest.raises(ValueError, match="workspace: holds"):
        q.ffn_f8(x, w13, s13, w2, s2, out=y, workspace=T((16,), U8))


def test_moe(q):
    e, h, i, k = 4, 256, 512, 2
    up, down = T((q.packed_bytes(q.SB4, e * 2 * i, h),), U8), T((q.packed_bytes(q.SB4, e * h, i),), U8)
    x, logits, y = T((N, h), F16), T((N, e), F32), T((N, h), F16)
    ids, w, work = T((N, k), I32), T((N, k), F32), T((1 << 20,), U8)
    out = dict(ids=ids, weights=w, out=y, workspace=work)

    def bad(exc, match, x=x, logits=logits, up=up, down=down, **change):
        with pytest.raises(exc, match=match):
            q.moe(q.SB4, x, logits, up, down, i, k, **(out | change))

    bad(TypeError, "x: element type", x=T((N, h), F32))
    bad(TypeError, "logits: element type", logits=T((N, e), F16))
    bad(ValueError, "rows for 3 tokens", logits=T((N + 1, e), F32))
    bad(ValueError, "4 columns for 5 experts", experts=5)
    bad(ValueError, "experts, ids and weights are needed", logits=None)
    bad(ValueError, "experts, ids and weights are needed", logits=None, experts=e, ids=None)
    bad(ValueError, "gate_up: holds", up=T((q.packed_bytes(q.SB4, e * 2 * i, h) - 1,), U8))
    bad(ValueError, "down: holds", down=T((q.packed_bytes(q.SB4, e * h, i) - 1,), U8))
    bad(ValueError, "ids: expected 6", ids=T((N, 1), I32))
    bad(TypeError, "ids: element type", ids=T((N, k), torch.int64))
    bad(ValueError, "weights: must be contiguous", weights=T((N, k), F32, contiguous=False))
    bad(ValueError, "out: expected 768", out=T((N, h + 256), F16))
    bad(ValueError, "workspace: holds", workspace=T((100,), U8))
    bad(ValueError, "other arguments", logits=T((N, e), F32, index=1))


def test_quantize_f8_out_of_another_shape(q):
    """The kernel writes the scales of w's shape, ceil(130/128) * 2 = 4 here; an `out` of as many
    elements in 260 rows of 128 has only 3, and the fourth would land behind them."""
    with pytest.raises(ValueError, match="out: expected shape"):
        q.quantize_f8(T((130, 256), F32), out=T((260, 128), F8), scale=T((3, 1), F32))
    with pytest.raises(ValueError, match="out: expected shape"):
        q.quantize_f8(T((128, 256), F32), out=T((256, 128), U8), scale=T((1, 2), F32))
    with pytest.raises(ValueError):
        q.quantize_f8(T((130, 256), F32), out=T((130 * 256,), F8), scale=T((2, 2), F32))


def test_moe_counts_past_32_bits(q):
    """experts and top_k cross the C boundary as 32-bit ints.  2^32 + 4 experts are more rows than
    any packed matrix holds, for which the byte count is 0, so a tensor of any size passed that
    check, and the library saw 4 experts."""
    tiny, big = T((16,), U8), 2 ** 32
    out = dict(ids=T((N, 2), I32), weights=T((N, 2), F32), out=T((N, 256), F16), workspace=T((1 << 20,), U8))
    with pytest.raises(ValueError, match="experts: 4294967300 is past"):
        q.moe(q.SB4, T((N, 256), F16), None, tiny, tiny, 512, 2, experts=big + 4, **out)
    with pytest.raises(ValueError, match="top_k: 4294967298 is past"):
        q.moe(q.SB4, T((N, 256), F16), T((N, 4), F32), tiny, tiny, 512, big + 2, **out)


def test_moe_scale_of_given_weights(q):
    """Weights of the caller's router are taken as they are: a scale for them is not dropped silently."""
    up, down = T((q.packed_bytes(q.SB4, 4 * 1024, 256),), U8), T((q.packed_bytes(q.SB4, 4 * 256, 512),), U8)
    out = dict(ids=T((N, 2), I32), weights=T((N, 2), F32), out=T((N, 256), F16), workspace=T((1 << 20,), U8))
    for scale in (2.0, 0.0, float("nan")):
        with pytest.raises(ValueError, match="weight_scale"):
            q.moe(q.SB4, T((N, 256), F16), None, up, down, 512, 2, experts=4, weight_scale=scale, **out)
