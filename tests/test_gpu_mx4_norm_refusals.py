"""What the bindings of the 4-bit rows, their products and the norm refuse: shapes, types, strides and
sizes that do not fit together.  Nothing is launched."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from combine_moe_route_gb300 import build
    build.build()
    return torch.device("cuda:0")


def test_four_bit_rows(gpu):
    import combine_moe_route_gb300 as moe
    x = torch.zeros((4, 64), device=gpu)
    q, s = moe.quantize_mx4(x)
    for call in (lambda: moe.quantize_mx4(x.half()), lambda: moe.quantize_mx4(x[:, :48].contiguous()),
                 lambda: moe.quantize_mx4(x[:, :32]), lambda: moe.quantize_mx4(x, out=q[:3]),
                 lambda: moe.quantize_mx4(x, out_scale=s.int()), lambda: moe.dequantize_mx4(q, s[:, :1].contiguous()),
                 lambda: moe.dequantize_mx4(q[:, :24].contiguous(), s), lambda: moe.dequantize_mx4(q.int(), s),
                 lambda: moe.dequantize_mx4(q, s, out=torch.empty((4, 64), device=gpu)),
                 lambda: moe.dequantize_mx4(q, None, out=torch.empty((4, 64), dtype=torch.bfloat16, device=gpu)),
                 lambda: moe.dequantize_mx4(q, s.cpu())):
        with pytest.raises(ValueError):
            call()


def test_products(gpu):
    import combine_moe_route_gb300 as moe
    a, sa = moe.quantize_mx4(torch.zeros((6, 64), device=gpu))
    w, sw = moe.quantize_mx4(torch.zeros((2, 64, 64), device=gpu))
    off = torch.tensor([0, 3, 6], dtype=torch.int32, device=gpu)
    good = dict(a=a, a_scale=sa, w=w, w_scale=sw, expert_offsets=off)
    for product in (moe.expert_gemm_mx4, moe.expert_gated_gemm_mx4):
        product(**good)
        for bad in (dict(a=a[:5]), dict(a=a.float()), dict(a=a[0]), dict(a_scale=sa[:, :1].contiguous()),
                    dict(a_scale=sa.int()), dict(w=w[0]), dict(w=w[:, :, :16].contiguous()), dict(w=w[:, ::2]),
                    dict(w_scale=sw[:, :32].contiguous()), dict(expert_offsets=off.long()),
                    dict(expert_offsets=off[:2]), dict(w_scale=sw.cpu()), dict(out=torch.empty((6, 63), device=gpu))):
            with pytest.raises(ValueError):
                product(**{**good, **bad})
    with pytest.raises(ValueError, match="out_dtype"):
        moe.expert_gemm_mx4(**good, out_dtype=torch.float16)
    w3, s3 = moe.quantize_mx4(torch.zeros((2, 32, 64), device=gpu))
    with pytest.raises(ValueError, match="multiple of 32"):
        moe.expert_gated_gemm_mx4(a, sa, w3, s3, off)
    w3, s3 = moe.quantize_mx4(torch.zeros((2, 24, 64), device=gpu))
    with pytest.raises(moe.MoeError):   # N not a multiple of 16
        moe.expert_gemm_mx4(a, sa, w3, s3, off)
    with pytest.raises(moe.MoeError):   # not at 16 bytes
        moe.expert_gemm_mx4(torch.zeros(6 * 32 + 8, dtype=torch.uint8, device=gpu)[8:].view(6, 32), sa, w, sw, off)


def test_norm(gpu):
    import combine_moe_route_gb300 as moe
    x, w = torch.zeros((4, 136), device=gpu, dtype=torch.bfloat16), torch.ones(136, device=gpu, dtype=torch.bfloat16)
    moe.rms_norm(x, w)
    for bad in (dict(x=x.float()), dict(x=x[0]), dict(x=x[:, :128]), dict(weight=w[:128]), dict(weight=w.float()),
                dict(residual=x[:3]), dict(residual=x.cpu()), dict(fp8=True), dict(eps=-1.0), dict(eps=float("nan")),
                dict(out=x.float()), dict(residual=x.clone(), out=x, out_h=x)):
        with pytest.raises(ValueError):
            moe.rms_norm(**{**dict(x=x, weight=w), **bad})
    with pytest.raises(moe.MoeError):   # H not a multiple of 8
        moe.rms_norm(torch.zeros((4, 12), device=gpu, dtype=torch.bfloat16), w[:12].contiguous())
    good = dict(dy=x, h=x, weight=w)
    moe.rms_norm_backward(**good)
    for bad in (dict(dy=x[:3]), dict(dy=x.float()), dict(h=x[:, :128]), dict(weight=w[:8]), dict(dh=x[0]),
                dict(eps=-1.0), dict(out=x.float()), dict(dweight=w), dict(workspace=torch.zeros(64, device=gpu))):
        with pytest.raises(ValueError):
            moe.rms_norm_backward(**{**good, **bad})
