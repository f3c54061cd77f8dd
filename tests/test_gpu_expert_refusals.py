"""The binding's refusals on CUDA tensors: shapes, types, layouts and devices that do not fit."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def t():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from combine_moe_route_gb300 import build
    build.build()
    dev = "cuda:0"
    e4 = torch.float8_e4m3fn
    return dict(a=torch.zeros((4, 128), dtype=e4, device=dev), sa=torch.zeros((4, 1), device=dev),
                w=torch.zeros((2, 256, 128), dtype=e4, device=dev), sw=torch.zeros((2, 2, 1), device=dev),
                off=torch.tensor([0, 2, 4], dtype=torch.int32, device=dev),
                x=torch.zeros((4, 128), dtype=torch.bfloat16, device=dev), k=torch.zeros((2, 2), device=dev),
                at=torch.arange(4, dtype=torch.int32, device=dev), idx=torch.zeros((2, 2), dtype=torch.int32, device=dev))


def test_products(t):
    import combine_moe_route_gb300 as moe
    a, sa, w, sw, off = (t[k] for k in ("a", "sa", "w", "sw", "off"))
    for call in (moe.expert_gemm, moe.expert_gated_gemm):
        for args in ((a.float(), sa, w, sw, off), (a, sa.double(), w, sw, off), (a, sa, w, sw.bfloat16(), off),
                     (a, sa, w, sw, off.long()), (a, sa, w, sw, off[:2]), (a, sa[:2], w, sw, off), (a, sa, w, sw[:1], off),
                     (a, sa, w[0], sw, off), (a[:, :112], sa, w, sw, off), (a, sa, w.transpose(1, 2), sw, off),
                     (a, sa.cpu(), w, sw, off)):
            with pytest.raises(ValueError):
                call(*args)
    with pytest.raises(ValueError):
        moe.expert_gemm(a, sa, w, sw, off, transpose=True)                      # contracts over 256
    with pytest.raises(ValueError):
        moe.expert_gemm(a, sa, w, sw, off, out_dtype=torch.float16)
    with pytest.raises(ValueError):
        moe.expert_gemm(a, sa, w, sw, off, out=torch.empty((4, 128), dtype=torch.bfloat16, device="cuda:0"))
    with pytest.raises(ValueError):
        moe.expert_gated_gemm(a, sa, w[:, :128].contiguous(), sw[:, :1].contiguous(), off)   # I = 64
    misaligned = torch.zeros(4 * 128 + 8, dtype=torch.uint8, device="cuda:0")[8:].view(4, 128)
    with pytest.raises(moe.MoeError):
        moe.expert_gemm(misaligned, sa, w, sw, off)


def test_gradients(t):
    import combine_moe_route_gb300 as moe
    x, k, at, idx = t["x"], t["k"], t["at"], t["idx"]
    for args in ((x, x, at, k), (x[:2].float(), x, at, k), (x[:2], x.float(), at, k), (x[:2], x, at.long(), k),
                 (x[:2], x, at[:3], k), (x[:2], x, at, k.double()), (x[:2], x, at, k[0])):
        with pytest.raises(ValueError):
            moe.combine_backward(*args)
    with pytest.raises(ValueError):
        moe.combine_backward(x[:2], x, at, k, topk_idx=idx)                     # no E
    with pytest.raises(ValueError):
        moe.combine_backward(x[:2], x, at, k, E=4)
    with pytest.raises(ValueError):
        moe.combine_backward(x[:2], x, at, k, dlogits=torch.empty((2, 4), device="cuda:0"))
    for bad in (0, 3):
        with pytest.raises(ValueError):
            moe.dispatch_backward(x, at, bad)
    with pytest.raises(ValueError):
        moe.dispatch_backward(x, at, 2, out_dtype=torch.float16)
    with pytest.raises(ValueError):
        moe.expert_gated_backward(x, x)
    with pytest.raises(moe.MoeError):
        moe.expert_gated_backward(x, x[:, :64].contiguous())                    # 64 channels do not make a block
