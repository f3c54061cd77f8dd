"""The whole layer with real experts, forward and backward, against the same chain in 64 bits on
the quantised values the GPU kernels exchange, and its gradients against differences."""
import numpy as np
import pytest
import torch

import _expert_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from combine_moe_route_gb300 import build
    build.build()
    return torch.device("cuda:0")


def _case(gpu, B, E, K, H, inner, seed):
    import combine_moe_route_gb300 as moe
    rng = np.random.default_rng(seed)
    T = sum(B)
    w = moe.ExpertWeights.quantized(
        torch.from_numpy(rng.standard_normal((E, 2 * inner, H)).astype(np.float32) / H ** 0.5).to(gpu),
        torch.from_numpy(rng.standard_normal((E, H, inner)).astype(np.float32) / inner ** 0.5).to(gpu))
    x = torch.from_numpy(rng.standard_normal((T, H)).astype(np.float32)).bfloat16()
    logits = torch.from_numpy(rng.standard_normal((T, E)).astype(np.float32))
    dout = torch.from_numpy(rng.standard_normal((T, H)).astype(np.float32)).bfloat16()
    return w, x, logits, dout


def _dense(w, scale):
    return ref._dequant_weight(w.cpu(), scale.cpu())


@pytest.mark.parametrize("B,E,K,H,inner", [([5, 0, 9, 2], 8, 2, 256, 128), ([33, 1], 4, 3, 384, 256),
                                           ([700], 2, 1, 128, 384), ([1], 16, 4, 640, 128)])
def test_layer(gpu, B, E, K, H, inner):
    import combine_moe_route_gb300 as moe
    w, x, logits, dout = _case(gpu, B, E, K, H, inner, H + inner)
    f = moe.expert_layer(x.to(gpu), logits.to(gpu), B, K, w, train=True, out_dtype=torch.float32)
    dx, dl = moe.expert_layer_backward(dout.to(gpu), f, w)
    # forward in 64 bits, every quantisation by the kernels' values up to one code
    T = sum(B)
    idx, at = f.topk_idx.long().cpu(), f.dispatch.tok2row.long().cpu().view(T, K)
    w13, w2, p = _dense(w.w13, w.w13_scale), _dense(w.w2, w.w2_scale), f.topk_w.double().cpu()
    xq = ref._dequant_rows(f.dispatch.recv_x.cpu(), f.dispatch.recv_scale.cpu())
    vq = ref._dequant_rows(f.gated.q.cpu(), f.gated.scale.cpu())
    out = torch.zeros((T, H), dtype=torch.float64)
    for t in range(T):
        for j in range(K):
            e, r = int(idx[t, j]), int(at[t, j])
            # one e4m3 step of 2^-3 on a block's largest value, halved by rounding
            assert (xq[r] - x[t].double()).abs().max() <= x[t].double().abs().max() * 2.0 ** -4
            h = w13[e] @ xq[r]
            v = ref.gate(h[:inner], h[inner:])
            assert (vq[r] - v).abs().max() <= v.abs().max() * 2.0 ** -4 * 1.01
            out[t] += p[t, j] * (w2[e] @ vq[r])
    # y is rounded to bf16 before the sum
    scale = out.abs().max() + f.y.double().cpu().abs().max()
    assert (f.out.cpu().double() - out).abs().max() <= 2.0 ** -8 * scale
    # backward: the chain of the kernels' own gradients is near the exact gradient of that forward.
    # Two quantisations to 3 fraction bits (relative error below 2^-4 each, 0.026 of the norm for
    # each on average) and bf16 roundings on the way
    exact = torch.zeros((T, H), dtype=torch.float64)
    dw = torch.zeros((T, K), dtype=torch.float64)
    for t in range(T):
        for j in range(K):
            e, r = int(idx[t, j]), int(at[t, j])
            h = w13[e] @ xq[r]
            dv = w2[e].T @ (p[t, j] * dout[t].double())
            dg, du, _ = ref.gate_grad(h[:inner], h[inner:], dv)
            exact[t] += w13[e].T @ torch.cat([dg, du])
            dw[t, j] = (w2[e] @ vq[r]) @ dout[t].double()
    assert (dx.cpu().double() - exact).norm() <= 0.08 * exact.norm()
    dlw = torch.zeros((T, E), dtype=torch.float64).scatter_(1, idx, p * (dw - (p * dw).sum(1, keepdim=True)))
    assert (dl.cpu().double() - dlw).abs().max() <= 2.0 ** -7 * (dlw.abs().max() + 1)


def test_layer_gradient_against_differences(gpu):
    """Directional differences of the 64-bit layer (without quantisation of its activations) agree
    with the gradients to the accuracy of e4m3."""
    import combine_moe_route_gb300 as moe
    B, E, K, H, inner = [6, 10], 8, 2, 256, 256
    w, x, logits, dout = _case(gpu, B, E, K, H, inner, 77)
    f = moe.expert_layer(x.to(gpu), logits.to(gpu), B, K, w, train=True)
    dx, dl = moe.expert_layer_backward(dout.to(gpu), f, w)
    idx = f.topk_idx.long().cpu()
    w13, w2 = _dense(w.w13, w.w13_scale), _dense(w.w2, w.w2_scale)

    def loss(xx, lg):
        p = torch.softmax(lg.gather(1, idx), 1)
        total = 0.0
        for t in range(16):
            for j in range(K):
                h = w13[idx[t, j]] @ xx[t]
                total += float(p[t, j] * (w2[idx[t, j]] @ ref.gate(h[:inner], h[inner:])) @ dout[t].double())
        return total

    rng = np.random.default_rng(1)
    x64, l64 = x.double(), logits.double()
    step = 1e-4
    for _ in range(3):
        v = torch.from_numpy(rng.standard_normal((16, H)))
        diff = (loss(x64 + step * v, l64) - loss(x64 - step * v, l64)) / (2 * step)
        # errors of 0.08 of each token's gradient, in directions of unit variance
        assert abs(float((dx.cpu().double() * v).sum()) - diff) <= 4 * 0.08 * float(dx.double().norm())
        u = torch.from_numpy(rng.standard_normal((16, E)))
        diff = (loss(x64, l64 + step * u) - loss(x64, l64 - step * u)) / (2 * step)
        assert abs(float((dl.cpu().double() * u).sum()) - diff) <= 4 * 0.08 * float(dl.double().norm()) + 1e-3


def test_serving_form_keeps_no_activations_and_trains_refuses(gpu):
    import combine_moe_route_gb300 as moe
    w, x, logits, dout = _case(gpu, [1], 8, 2, 256, 128, 5)
    f = moe.expert_layer(x.to(gpu), logits.to(gpu), [1], 2, w)
    assert f.gated.h is None and f.out.dtype == torch.bfloat16
    with pytest.raises(ValueError, match="train"):
        moe.expert_layer_backward(dout.to(gpu), f, w)


def test_layer_in_a_graph_and_on_a_stream(gpu):
    import combine_moe_route_gb300 as moe
    w, x, logits, dout = _case(gpu, [40, 24], 8, 2, 256, 128, 6)
    x, logits, dout = x.to(gpu), logits.to(gpu), dout.to(gpu)
    f = moe.expert_layer(x, logits, [40, 24], 2, w, train=True)
    dx, dl = moe.expert_layer_backward(dout, f, w)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        f2 = moe.expert_layer(x, logits, [40, 24], 2, w, train=True)
        dx2, dl2 = moe.expert_layer_backward(dout, f2, w)
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(f2.out, f.out) and torch.equal(dx2, dx) and torch.equal(dl2, dl)


def test_example_runs(gpu):
    import subprocess
    import sys
    r = subprocess.run([sys.executable, "-m", "combine_moe_route_gb300.experts"], capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0, r.stderr
    assert "device status 0, 0" in r.stdout
