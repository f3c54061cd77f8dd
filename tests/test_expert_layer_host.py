"""Quantisation of weights by blocks (runs on the CPU) and the package's lazy names."""
import torch


def test_quantize_blocks():
    from combine_moe_route_gb300 import quantize_blocks
    gen = torch.Generator().manual_seed(0)
    w = torch.randn((3, 208, 400), generator=gen)
    w[1, :128, :128] = 0
    q, s = quantize_blocks(w)
    assert q.shape == w.shape and s.shape == (3, 2, 4) and q.dtype == torch.float8_e4m3fn
    full = s.repeat_interleave(128, 1)[:, :208].repeat_interleave(128, 2)[:, :, :400]
    # half an e4m3 step: 2^-4 of the value, or 2^-10 of a block's scale below the normal range
    assert ((q.float() * full - w).abs() <= w.abs() * 2.0 ** -4 * 1.0001 + full * 2.0 ** -10).all()
    assert torch.isfinite(s).all() and (s > 0).all()
    for e in range(3):
        for n in range(2):
            for c in range(4):
                block = w[e, 128 * n:128 * n + 128, 128 * c:128 * c + 128]
                if block.abs().max() > 0:
                    assert float(q[e, 128 * n:128 * n + 128, 128 * c:128 * c + 128].float().abs().max()) == 448.0


def test_package_names():
    import combine_moe_route_gb300 as moe
    for name in moe.__all__:
        assert getattr(moe, name) is not None, name
    assert callable(moe.expert_layer) and callable(moe.expert_gemm)
