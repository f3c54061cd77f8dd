"""GPU tests of a layer with 4-bit experts and of the block around a layer (residual, norm, router),
each step against 64-bit references of the step's own inputs, on streams and in a graph."""
import numpy as np
import pytest
import torch

import _expert_ref as eref
import _mx4_ref as ref

pytestmark = pytest.mark.gpu
T, H, I, E, K, B = 203, 512, 160, 8, 3, [100, 0, 100, 3]


@pytest.fixture(scope="module")
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from combine_moe_route_gb300 import build
    build.build()
    return torch.device("cuda:0")


def _inputs(gpu, inner=I):
    gen = torch.Generator(device=gpu).manual_seed(3)

    def rand(*shape):
        return torch.randn(shape, generator=gen, device=gpu)

    return dict(x=rand(T, H).bfloat16(), res=rand(T, H).bfloat16(), norm=(1 + 0.2 * rand(H)).bfloat16(),
                router=rand(E, H) / H ** 0.5, w13=rand(E, 2 * inner, H) / H ** 0.5, w2=rand(E, H, inner) / inner ** 0.5)


def test_four_bit_layer_step_by_step(gpu):
    import combine_moe_route_gb300 as moe
    d = _inputs(gpu)
    w = moe.ExpertWeightsMx4.quantized(d["w13"], d["w2"])
    codes, byte = ref.quantize(d["w13"].cpu().double())
    assert torch.equal(w.w13.cpu(), ref.pack(codes)) and torch.equal(w.w13_scale.cpu(), byte) and w.E == E
    logits = d["x"].float() @ d["router"].T
    f = moe.expert_layer(d["x"], logits, B, K, w)
    off = f.dispatch.expert_offsets.cpu()
    codes, byte = ref.quantize(f.dispatch.recv_x.cpu().double())
    inp = dict(a=ref.pack(codes), a_scale=byte, w=w.w13.cpu(), w_scale=w.w13_scale.cpu(), off=off)
    p, mag = ref.product(inp)
    err = ref.product_bound(mag, H)
    g, u, eg, eu = p[:, :I], p[:, I:], err[:, :I], err[:, I:]
    v = eref.gate(g, u)
    bound = 1.1 * eg * (u.abs() + eu) + (g.abs() + eg) * eu + 16 * 2.0 ** -24 * v.abs()
    assert ref.quantized_ok(f.gated.q.cpu(), f.gated.scale.cpu(), v, bound) == (True, True)
    inp = dict(a=f.gated.q.cpu(), a_scale=f.gated.scale.cpu(), w=w.w2.cpu(), w_scale=w.w2_scale.cpu(), off=off)
    y, mag = ref.product(inp)
    assert ((f.y.cpu().double() - y).abs() <= ref.product_bound(mag, I) + 2.0 ** -8 * y.abs()).all()
    assert torch.equal(f.out, moe.combine(f.y, f.dispatch.tok2row, f.topk_w))
    assert moe.get_expert_error()[0] == 0


def test_four_bit_layer_refuses_training(gpu):
    import combine_moe_route_gb300 as moe
    d = _inputs(gpu)
    w = moe.ExpertWeightsMx4.quantized(d["w13"], d["w2"])
    logits = d["x"].float() @ d["router"].T
    with pytest.raises(ValueError, match="no gradient"):
        moe.expert_layer(d["x"], logits, B, K, w, train=True)
    f = moe.expert_layer(d["x"], logits, B, K, w)
    with pytest.raises(ValueError, match="pre-activations"):
        moe.expert_layer_backward(d["x"], f, w)
    with pytest.raises(ValueError, match="a column for each"):
        moe.expert_layer(d["x"], logits[:, :4].contiguous(), B, K, w)


@pytest.mark.parametrize("residual", [False, True])
def test_block(gpu, residual):
    """Forward: the norm's rows and the layer on them.  Backward: the chain's formulas at the values
    that each step got."""
    import combine_moe_route_gb300 as moe
    d = _inputs(gpu, 128)
    w = moe.ExpertWeights.quantized(d["w13"], d["w2"])
    res = d["res"] if residual else None
    f = moe.expert_block(d["x"], res, d["norm"], d["router"], B, K, w, train=True)
    n = moe.rms_norm(d["x"], d["norm"], residual=res)
    assert torch.equal(f.h, n.h) and torch.equal(f.y, n.y)
    layer = moe.expert_layer(n.y, f.logits, B, K, w, train=True)
    assert torch.equal(f.out, layer.out)
    want = n.y.double() @ d["router"].double().T
    assert ((f.logits.double() - want).abs() <= H * 2.0 ** -23 * (n.y.double().abs() @ d["router"].double().abs().T)).all()

    gen = torch.Generator(device=gpu).manual_seed(4)
    dout = torch.randn((T, H), generator=gen, device=gpu).bfloat16()
    dh = torch.randn((T, H), generator=gen, device=gpu).bfloat16() if residual else None
    g = moe.expert_block_backward(dout, dh, f, d["norm"], d["router"], w)
    dy, dlogits = moe.expert_layer_backward(dout, f.layer, w)
    dl = dlogits.double()
    err = T * 2.0 ** -23 * (dl.abs().T @ f.y.double().abs())
    assert ((g.drouter.double() - dl.T @ f.y.double()).abs() <= err).all()
    dy64 = dy.double() + dl @ d["router"].double()
    # dy is rounded to bf16 between the two; then the norm's own gradient of that
    h64, n64 = f.h.double(), None
    r = 1 / torch.sqrt((h64 * h64).mean(1, keepdim=True) + 1e-6)
    n64, gw = h64 * r, dy64 * d["norm"].double()
    dx = r * (gw - n64 * (gw * n64).mean(1, keepdim=True)) + (dh.double() if residual else 0)
    step = 2.0 ** -8 * 1.01   # of dy's rounding, and room for fp32's
    slack = step * r * (gw.abs() + n64.abs() * (gw * n64).abs().mean(1, keepdim=True))
    assert ((g.dx.double() - dx).abs() <= slack + 2.0 ** -8 * (dx.abs() + slack)).all()
    assert ((g.dnorm.double() - (dy64 * n64).sum(0)).abs() <= step * (dy64 * n64).abs().sum(0)).all()


def test_block_on_another_stream_and_in_a_graph(gpu):
    import combine_moe_route_gb300 as moe
    d = _inputs(gpu, 128)
    w, four = moe.ExpertWeights.quantized(d["w13"], d["w2"]), moe.ExpertWeightsMx4.quantized(d["w13"], d["w2"])
    dout = d["res"].clone()

    def run(stream=None):
        f = moe.expert_block(d["x"], d["res"], d["norm"], d["router"], B, K, w, train=True, stream=stream)
        g = moe.expert_block_backward(dout, dout, f, d["norm"], d["router"], w, stream=stream)
        m = moe.expert_block(f.out, f.h, d["norm"], d["router"], B, K, four, stream=stream)
        return f.out, g.dx, g.dnorm, g.drouter, m.out

    want = run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = run(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    for seed in (1, 2):
        gen = torch.Generator(device=gpu).manual_seed(seed)
        d["x"].copy_(torch.randn((T, H), generator=gen, device=gpu))
        graph.replay()
        got = [t.clone() for t in out]
        assert all(torch.equal(a, b) for a, b in zip(got, run()))
    assert moe.get_expert_error()[0] == 0
