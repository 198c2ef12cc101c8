"""The binding's refusals for the microscaling formats and the norm (CPU only):
every bad argument raises before a compute entry point is reached."""
import pytest
import torch

from test_binding_checks import FakeGpuTensor, RecordingLib, pytestmark  # noqa: F401

F32, F16, BF16, U8 = torch.float32, torch.float16, torch.bfloat16, torch.uint8
F8, E8 = torch.float8_e4m3fn, torch.float8_e8m0fnu
M, K, N = 200, 256, 3


class Lib(RecordingLib):
    GEOMETRY = RecordingLib.GEOMETRY + ("qblk_gemm_mxfp4_workspace", "qblk_linear_mxfp4_workspace")


@pytest.fixture()
def q(monkeypatch):
    import bit_block_quant_amd as q
    rec = Lib(q._lib)
    monkeypatch.setattr(q, "_lib", rec)
    yield q
    assert rec.calls == [], f"a compute entry point was reached: {rec.calls}"


T = FakeGpuTensor
WQ, WS = T((M, K // 2), U8), T((M, K // 32), E8)


def test_quantizers(q):
    for f in (q.quantize_mxfp4, q.quantize_mxfp8):
        with pytest.raises(ValueError, match="GPU tensor"):
            f(torch.zeros(M, K))
        with pytest.raises(ValueError, match="multiple of 32"):
            f(T((M, 40), F32))
        with pytest.raises(ValueError, match="contiguous"):
            f(T((M, K), F16, contiguous=False))
        with pytest.raises(ValueError, match="dimensions"):
            f(T((M * K,), F16))
        with pytest.raises(TypeError, match="element type"):
            f(T((M, K), F8))
    with pytest.raises(ValueError, match="out: expected shape"):
        q.quantize_mxfp4(T((M, K), F32), out=T((M, K), U8), scale=WS)
    with pytest.raises(ValueError, match="out: expected shape"):
        q.quantize_mxfp4(T((M, K), F32), out=T((2 * M, K // 4), U8), scale=WS)
    with pytest.raises(TypeError, match="out: element type"):
        q.quantize_mxfp4(T((M, K), F32), out=T((M, K // 2), F8), scale=WS)
    with pytest.raises(ValueError, match="scale: expected 1600"):
        q.quantize_mxfp4(T((M, K), F32), out=WQ, scale=T((M, 4), E8))
    with pytest.raises(TypeError, match="scale: element type"):
        q.quantize_mxfp8(T((M, K), F32), out=T((M, K), F8), scale=T((M, 8), F32))
    with pytest.raises(ValueError, match="other arguments"):
        q.quantize_mxfp8(T((M, K), F32), out=T((M, K), F8, index=1), scale=WS)


def test_dequant(q):
    with pytest.raises(ValueError, match="scale: expected 1600"):
        q.dequant_mx(WQ, T((M, 7), E8), out=T((M, K), F32))
    with pytest.raises(ValueError, match="multiple of 32"):
        q.dequant_mx(T((M, 8), U8), T((M, 1), E8), out=T((M, 16), F32))
    with pytest.raises(TypeError, match="element type"):
        q.dequant_mx(T((M, K), F16), WS, out=T((M, K), F32))
    with pytest.raises(ValueError, match="expected 51200 elements"):
        q.dequant_mx(WQ, WS, out=T((M, K // 2), F32))


def test_products(q):
    x, y = T((N, K), BF16), T((N, M), BF16)
    with pytest.raises(ValueError, match="columns"):
        q.linear_mxfp4(T((N, 128), BF16), WQ, WS, out=y)
    with pytest.raises(ValueError, match="act: expected"):
        q.linear_mxfp4(x, WQ, WS, act=q.ACT_F8, out=y)
    with pytest.raises(ValueError, match="act: expected"):
        q.linear_mxfp4(x, WQ, WS, act="mxfp4", out=y)
    with pytest.raises(ValueError, match="scale: expected 1600"):
        q.linear_mxfp4(x, WQ, T((M, 2), E8), out=y)
    with pytest.raises(TypeError, match="element type"):
        q.linear_mxfp4(x, T((M, K // 2), F8), WS, out=y)
    with pytest.raises(ValueError, match="expected 600 elements"):
        q.linear_mxfp4(x, WQ, WS, out=T((N, M + 1), BF16))
    with pytest.raises(ValueError, match="workspace: holds"):
        q.linear_mxfp4(T((70, K), BF16), WQ, WS, out=T((70, M), BF16), workspace=T((16,), U8))
    xq, xs = T((N, K), F8), T((N, K // 32), E8)
    with pytest.raises(ValueError, match="xq scale: expected 24"):
        q.gemm_mxfp4(WQ, WS, xq, T((N,), E8), out=T((N, M), F32))
    with pytest.raises(ValueError, match="512 columns, wq has 256"):
        q.gemm_mxfp4(WQ, WS, T((N, K), U8), T((N, 16), E8), out=T((N, M), F32))
    with pytest.raises(TypeError, match="xq: element type"):
        q.gemm_mxfp4(WQ, WS, T((N, K), F16), xs, out=T((N, M), F32))
    with pytest.raises(ValueError, match="other arguments"):
        q.gemm_mxfp4(WQ, WS, T((N, K), F8, index=1), xs, out=T((N, M), F32))


def test_norm(q):
    x, w = T((N, K), BF16), T((K,), F32)
    out = dict(out=T((N, K), F8), scale=T((N, 2), F32))

    def bad(exc, match, x=x, w=w, **change):
        with pytest.raises(exc, match=match):
            q.rmsnorm(x, w, **(out | change))

    bad(ValueError, "GPU tensor", x=torch.zeros(N, K))
    bad(TypeError, "x: element type", x=T((N, K), F8))
    bad(ValueError, "quant: expected", quant=4)
    bad(ValueError, "quant: expected", quant="f8")
    bad(ValueError, "multiple of 128", x=T((N, 160), BF16))
    bad(ValueError, "multiple of 32", x=T((N, 144), BF16), quant=q.ACT_MXFP4)
    bad(ValueError, "multiple of 8", x=T((N, 12), BF16), quant=q.ACT_I8)
    bad(ValueError, "eps must not be", eps=-1.0)
    bad(ValueError, "eps must not be", eps=float("nan"))
    bad(ValueError, "weight: expected 256", w=T((K + 1,), F32))
    bad(TypeError, "residual: element type", residual=T((N, K), F32))
    bad(ValueError, "residual: expected 768", residual=T((1, K), BF16))
    bad(ValueError, "no residual", total=T((N, K), BF16))
    bad(ValueError, "total: expected 768", residual=x, total=T((N + 1, K), BF16))
    bad(TypeError, "total: element type", residual=x, total=T((N, K), F32))
    bad(ValueError, "nothing is quantized", quant=None)
    bad(ValueError, "out: expected shape", out=T((N, K // 2), F8))
    bad(ValueError, "scale: expected 6", scale=T((N,), F32))
    bad(TypeError, "scale: element type", quant=q.ACT_MXFP8)
    bad(TypeError, "out: element type", quant=q.ACT_I8, scale=T((N,), F32))
    bad(TypeError, "y: element type", y=T((N, K), F32))
    bad(ValueError, "y: expected 768", y=T((N, K - 8), BF16))
    bad(ValueError, "other arguments", y=T((N, K), BF16, index=1))
