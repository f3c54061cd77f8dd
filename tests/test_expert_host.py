"""Refusals of the expert products and the gradients, without a GPU: the C entries' validation
(nothing is enqueued) and the binding's checks of shapes, types and devices."""
import numpy as np
import pytest
import torch

OK, INVALID, UNSUPPORTED = 0, 1, 2
BF16, FP8, FP32 = 0, 1, 2
FAKE, ODD = 0x100000, 0x100008      # never dereferenced: every call below is refused or has nothing to do


@pytest.fixture(scope="module")
def lib():
    from combine_moe_route_gb300 import binding, build
    build.build()
    return binding.load_library()


def test_expert_gemm(lib):
    def call(E=4, N=256, C=256, rows=8, transpose=0, dtype=BF16, a=FAKE, sa=FAKE, w=FAKE, sw=FAKE, off=FAKE, out=FAKE):
        return lib.moe_expert_gemm(a, sa, w, sw, off, E, N, C, rows, transpose, dtype, out, None)

    for bad in (dict(E=0), dict(E=1025), dict(N=8), dict(N=0), dict(C=24), dict(C=-16), dict(N=65552), dict(rows=-1),
                dict(dtype=FP8), dict(dtype=7), dict(a=None), dict(sa=None), dict(w=None), dict(sw=None),
                dict(off=None), dict(out=None)):
        assert call(**bad) == INVALID, bad
        assert call(transpose=1, **bad) == INVALID, bad
    for odd in ("a", "w", "out"):
        assert call(**{odd: ODD}) == UNSUPPORTED
    assert call(rows=0, a=None, out=None) == OK


def test_expert_gated_gemm(lib):
    def call(E=4, I=256, C=256, rows=8, a=FAKE, sa=FAKE, w=FAKE, sw=FAKE, off=FAKE, q=FAKE, s=FAKE, h=None):
        return lib.moe_expert_gated_gemm(a, sa, w, sw, off, E, I, C, rows, q, s, h, None)

    for bad in (dict(E=0), dict(I=64), dict(I=192), dict(I=32896), dict(C=8), dict(rows=-2), dict(a=None),
                dict(sa=None), dict(w=None), dict(sw=None), dict(off=None), dict(q=None), dict(s=None)):
        assert call(**bad) == INVALID, bad
    for odd in ("a", "w", "q", "h"):
        assert call(**{odd: ODD}) == UNSUPPORTED
    assert call(rows=0, a=None, q=None) == OK


def test_expert_gated_backward(lib):
    def call(rows=8, I=256, dtype=BF16, h=FAKE, dv=FAKE, dh=FAKE, s=FAKE):
        return lib.moe_expert_gated_backward(h, dv, rows, I, dtype, dh, s, None)

    for bad in (dict(rows=-1), dict(I=0), dict(I=12), dict(I=136, dtype=FP8), dict(dtype=FP32), dict(h=None),
                dict(dv=None), dict(dh=None), dict(dtype=FP8, s=None)):
        assert call(**bad) == INVALID, bad
    for odd in ("h", "dv", "dh"):
        assert call(**{odd: ODD}) == UNSUPPORTED
    assert call(rows=0, h=None) == OK


def test_combine_backward(lib):
    def call(T=4, K=2, H=256, rows=8, E=16, dtype=BF16, dout=FAKE, y=FAKE, at=FAKE, w=FAKE, idx=FAKE, dy=FAKE, s=FAKE,
             dw=FAKE, dl=FAKE):
        return lib.moe_combine_backward(dout, y, at, w, idx, T, K, H, rows, E, dtype, dy, s, dw, dl, None)

    for bad in (dict(T=-1), dict(K=0), dict(K=33), dict(H=4), dict(H=20), dict(H=16392), dict(rows=-1),
                dict(rows=2 ** 31), dict(T=2 ** 30, K=2), dict(dtype=FP32), dict(H=264, dtype=FP8), dict(E=0),
                dict(E=1025), dict(dout=None), dict(y=None), dict(w=None), dict(idx=None), dict(dy=None),
                dict(dtype=FP8, s=None), dict(dw=None)):
        assert call(**bad) == INVALID, bad
    for odd in ("dout", "y", "dy"):
        assert call(**{odd: ODD}) == UNSUPPORTED
    assert call(T=0, dout=None) == OK


def test_dispatch_backward(lib):
    def call(T=4, K=2, H=256, rows=8, dtype=BF16, d=FAKE, at=FAKE, dx=FAKE):
        return lib.moe_dispatch_backward(d, at, T, K, H, rows, dtype, dx, None)

    for bad in (dict(T=-1), dict(K=0), dict(K=33), dict(H=12), dict(rows=-1), dict(rows=2 ** 31), dict(dtype=FP8),
                dict(d=None), dict(at=None), dict(dx=None)):
        assert call(**bad) == INVALID, bad
    for odd in ("d", "dx"):
        assert call(**{odd: ODD}) == UNSUPPORTED
    assert call(T=0, d=None) == OK


def test_binding_refuses_cpu_tensors():
    import combine_moe_route_gb300 as moe
    q, s = torch.zeros((4, 128), dtype=torch.float8_e4m3fn), torch.zeros((4, 1))
    w, sw = torch.zeros((2, 256, 128), dtype=torch.float8_e4m3fn), torch.zeros((2, 2, 1))
    off = torch.tensor([0, 2, 4], dtype=torch.int32)
    x, k = torch.zeros((4, 128), dtype=torch.bfloat16), torch.zeros((2, 2))
    at = torch.arange(4, dtype=torch.int32)
    for call in (lambda: moe.expert_gemm(q, s, w, sw, off), lambda: moe.expert_gated_gemm(q, s, w, sw, off),
                 lambda: moe.expert_gated_backward(x, x[:, :64].contiguous()),
                 lambda: moe.combine_backward(x[:2], x, at, k), lambda: moe.dispatch_backward(x, at, 2)):
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()


def test_reference_quantisation_agrees_with_the_oracle(oracle):
    """The fp32 rule the gradient tests compare with gives the oracle's bytes and scales."""
    import _expert_ref as ref
    from combine_moe_route_gb300 import workloads as wl
    rng = np.random.default_rng(0)
    x = torch.from_numpy((rng.standard_normal((5, 256)) * 3).astype(np.float32)).bfloat16()
    x[2, :128] = 0
    d = oracle.dispatch(wl.bf16_bits(x), np.zeros((5, 1), np.int32), [5], 1, fp8=True)
    q, s = ref.quantize_f32(x.float())
    assert np.array_equal(q.view(torch.uint8).numpy(), np.asarray(d["recv"]).view(np.uint8).reshape(5, 256))
    assert np.array_equal(s.numpy(), np.asarray(d["recv_scale"]).reshape(5, 2))
