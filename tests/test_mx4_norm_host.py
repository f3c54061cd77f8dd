"""Refusals of the 4-bit rows, their products and the norm, without a GPU, and the 64-bit references
the GPU tests compare with."""
import numpy as np
import pytest
import torch

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 4
BF16, FP8, FP32 = 0, 1, 2
FAKE, ODD = 0x100000, 0x100008      # never dereferenced: every call below is refused or has nothing to do


@pytest.fixture(scope="module")
def lib():
    from combine_moe_route_gb300 import binding, build
    build.build()
    return binding.load_library()


def test_quantize(lib):
    def call(x=FAKE, dtype=BF16, rows=4, C=64, q=FAKE, s=ODD):
        return lib.moe_quantize_mx4(x, dtype, rows, C, q, s, None)

    for bad in (dict(C=0), dict(C=16), dict(C=48), dict(C=-32), dict(rows=-1), dict(rows=2 ** 40), dict(dtype=FP8),
                dict(x=None), dict(q=None), dict(s=None)):
        assert call(**bad) == INVALID, bad
    for odd in ("x", "q"):
        assert call(**{odd: ODD}) == UNSUPPORTED
    assert call(rows=0, x=None, q=None, s=None) == OK


def test_dequantize(lib):
    def call(q=FAKE, s=ODD, rows=4, C=64, dtype=BF16, out=FAKE):
        return lib.moe_dequantize_mx4(q, s, rows, C, dtype, out, None)

    for bad in (dict(C=0), dict(C=33), dict(rows=-1), dict(rows=2 ** 40), dict(dtype=FP32), dict(dtype=FP8),
                dict(s=None), dict(q=None), dict(out=None)):
        assert call(**bad) == INVALID, bad
    for odd in ("q", "out"):
        assert call(**{odd: ODD}) == UNSUPPORTED
    assert call(rows=0, q=None) == OK


def test_products(lib):
    def call(E=4, N=256, C=256, rows=8, dtype=BF16, a=FAKE, sa=ODD, w=FAKE, sw=ODD, off=FAKE, out=FAKE):
        return lib.moe_expert_gemm_mx4(a, sa, w, sw, off, E, N, C, rows, dtype, out, None)

    for bad in (dict(E=0), dict(E=1025), dict(N=8), dict(N=0), dict(N=24), dict(C=16), dict(C=48), dict(C=-32),
                dict(N=65552), dict(C=65568), dict(rows=-1), dict(dtype=FP8), dict(a=None), dict(sa=None),
                dict(w=None), dict(sw=None), dict(off=None), dict(out=None)):
        assert call(**bad) == INVALID, bad
    for odd in ("a", "w", "out"):
        assert call(**{odd: ODD}) == UNSUPPORTED
    assert call(rows=0, a=None, out=None) == OK

    def gated(E=4, I=256, C=256, rows=8, a=FAKE, sa=ODD, w=FAKE, sw=ODD, off=FAKE, q=FAKE, s=ODD):
        return lib.moe_expert_gated_gemm_mx4(a, sa, w, sw, off, E, I, C, rows, q, s, None)

    for bad in (dict(E=0), dict(I=16), dict(I=48), dict(I=32800), dict(C=16), dict(rows=-2), dict(a=None),
                dict(sa=None), dict(w=None), dict(sw=None), dict(off=None), dict(q=None), dict(s=None)):
        assert gated(**bad) == INVALID, bad
    for odd in ("a", "w", "q"):
        assert gated(**{odd: ODD}) == UNSUPPORTED
    assert gated(rows=0, a=None, q=None) == OK


def test_norm(lib):
    def call(x=FAKE, res=FAKE, w=FAKE, T=4, H=256, eps=1e-6, y=FAKE, h=FAKE, q=None, s=None):
        return lib.moe_rms_norm(x, res, w, T, H, eps, y, h, q, s, None)

    nan = float("nan")
    for bad in (dict(T=-1), dict(H=4), dict(H=12), dict(H=16392), dict(eps=-1.0), dict(eps=nan), dict(x=None),
                dict(w=None), dict(y=None), dict(h=None), dict(res=None), dict(q=FAKE), dict(q=FAKE, s=FAKE, H=264)):
        assert call(**bad) == INVALID, bad
    for odd in ("x", "res", "w", "y", "h"):
        assert call(**{odd: ODD}) == UNSUPPORTED
    assert call(q=ODD, s=FAKE) == UNSUPPORTED
    assert call(T=0, x=None) == OK


def test_norm_backward(lib):
    def call(dy=FAKE, h=FAKE, w=FAKE, dh=FAKE, T=4, H=256, eps=1e-6, dx=FAKE, dw=FAKE, ws=FAKE, n=1 << 30):
        return lib.moe_rms_norm_backward(dy, h, w, dh, T, H, eps, dx, dw, ws, n, None)

    for bad in (dict(T=-1), dict(H=4), dict(H=12), dict(H=16392), dict(eps=-1.0), dict(dy=None), dict(h=None),
                dict(w=None), dict(dx=None), dict(dw=None)):
        assert call(**bad) == INVALID, bad
    need = lib.moe_rms_norm_workspace_bytes(4000, 2048)
    assert need >= 2048 * 4
    assert call(T=4000, H=2048, n=need - 1) == WORKSPACE and call(T=4000, H=2048, ws=None) == WORKSPACE
    assert lib.moe_rms_norm_workspace_bytes(4, 256) == 0
    for odd in ("dy", "h", "w", "dh", "dx", "ws"):
        assert call(**{odd: ODD}) == UNSUPPORTED
    assert lib.moe_rms_norm_workspace_bytes(0, 256) == 0 == lib.moe_rms_norm_workspace_bytes(4, 20)


def test_binding_refuses_cpu_tensors():
    import combine_moe_route_gb300 as moe
    q, s = torch.zeros((4, 32), dtype=torch.uint8), torch.zeros((4, 2), dtype=torch.uint8)
    w, sw = torch.zeros((2, 64, 32), dtype=torch.uint8), torch.zeros((2, 64, 2), dtype=torch.uint8)
    off = torch.tensor([0, 2, 4], dtype=torch.int32)
    x, g = torch.zeros((4, 64), dtype=torch.bfloat16), torch.zeros(64, dtype=torch.bfloat16)
    for call in (lambda: moe.quantize_mx4(x), lambda: moe.dequantize_mx4(q, s), lambda: moe.rms_norm(x, g),
                 lambda: moe.rms_norm_backward(x, x, g), lambda: moe.expert_gemm_mx4(q, s, w, sw, off),
                 lambda: moe.expert_gated_gemm_mx4(q, s, w, sw, off)):
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()


def test_reference_quantisation():
    """The 64-bit reference on values worked out by hand, and what it calls a right quantisation."""
    import _mx4_ref as ref
    v = torch.zeros(1, 64, dtype=torch.float64)
    v[0, :8] = torch.tensor([7.0, 5.0, -0.25, 0.75, -2.5, 3.5, 0.0, -0.0])
    v[0, 32] = 2.0 ** -126
    codes, byte = ref.quantize(v)
    assert byte.tolist() == [[127, 0]]
    assert codes[0, :8].tolist() == [7, 6, 8, 2, 8 + 4, 6, 0, 8]
    assert codes[0, 32].item() == 4                     # 2^-126 in units of 2^-127
    assert torch.equal(ref.unpack(ref.pack(codes)), codes)
    rng = np.random.default_rng(0)
    x = torch.from_numpy(rng.standard_normal((6, 96)))
    codes, byte = ref.quantize(x)
    none = torch.zeros_like(x)
    assert ref.quantized_ok(ref.pack(codes), byte, x, none) == (True, True)
    assert ref.quantized_ok(ref.pack(codes), byte + 1, x, none)[0] is False
    codes[2, 5] ^= 6
    assert ref.quantized_ok(ref.pack(codes), byte, x, none)[1] is False
