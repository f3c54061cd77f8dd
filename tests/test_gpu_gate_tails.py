"""Gates so negative that 1 + exp(-g) is near or past the largest fp32 value, and gates so positive
that it is 1: silu is as small as it is there, not zero, and counts where the other factor is large;
its gradient is, but for a logistic function below 2^-126, which counts as zero."""
import numpy as np
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


def test_forward(gpu):
    """Gates of -80 to -103 against up projections of 1e30: one channel carries both, so that a
    row's block holds one value 128 times and its scale is that value / 448."""
    from combine_moe_route_gb300 import binding as b
    I = C = 128
    scale = torch.arange(80, 103.25, 0.25) / 352          # of a row: the gate is -352 times it
    rows = scale.numel()
    a, w = torch.zeros((rows, C)), torch.zeros((1, 2 * I, C))
    a[:, 0], w[0, :I, 0], w[0, I:, 0] = 1.0, -352.0, 4.0
    up = np.float32(1e30)
    r = b.expert_gated_gemm(a.to(torch.float8_e4m3fn).to(gpu), scale.view(rows, 1).to(gpu),
                            w.to(torch.float8_e4m3fn).to(gpu), torch.tensor([[[1.0], [float(up)]]], device=gpu),
                            torch.tensor([0, rows], dtype=torch.int32, device=gpu))
    g, u = -352 * scale.double(), 4 * scale.double() * float(up)
    want = (g * u / (1 + torch.exp(-g))).abs()
    # g is rounded once (2^-24 of it, and so many relative errors of exp(g)); u, the exponential,
    # the division and three products take fewer than 16 roundings; below the normal numbers
    # exp(g) and the quotient are multiples of 2^-149 (a rounding each)
    err = want * 2.0 ** -24 * (g.abs() + 16) + 2 * 2.0 ** -149 * g.abs() * u
    got = r.scale.cpu().double().view(rows) * 448
    assert ((got - want).abs() <= err).all()
    big = want > 1e-10
    assert big.sum() > 60 and (r.q.float().cpu().abs()[big] == 448).all()


def test_gradient(gpu):
    from combine_moe_route_gb300 import binding as b
    g = torch.arange(-104, -79, 0.5).bfloat16().double()
    n = g.numel()
    I = 64
    u = torch.tensor(1e30).bfloat16().double()
    h = torch.zeros((1, 2 * I))
    h[0, :n], h[0, I:I + n] = g.float(), float(u)
    dv = torch.ones((1, I)).bfloat16()
    dh, _ = b.expert_gated_backward(h.bfloat16().to(gpu), dv.to(gpu), fp8=False)
    dg, du = dh[0, :n].cpu().double(), dh[0, I:I + n].cpu().double()
    s = torch.exp(g) / (1 + torch.exp(g))
    # a bf16 rounding (2^-8), the exponential's 2 + 1.2 |g| units of 2^-23 and a few roundings more;
    # s counts as zero below 2^-126, or is rounded to a multiple of 2^-149 there
    rel = 2.0 ** -8 + 2.0 ** -23 * (16 + 2 * g.abs())
    lost = torch.where(s < 2.0 ** -125, s.clamp(max=2.0 ** -126), 2.0 ** -149)
    wg, wu = u * s * (1 + g * (1 - s)), g * s
    assert ((dg - wg).abs() <= wg.abs() * rel + u * (1 + g.abs()) * lost).all()
    assert ((du - wu).abs() <= wu.abs() * rel + g.abs() * lost + 2.0 ** -134).all()
    assert (dg[g > -87] != 0).all()


def test_gradient_of_large_positive_gates(gpu):
    """The slope there is 1 whatever the gate: nothing of 1 - s is left to multiply it with."""
    from combine_moe_route_gb300 import binding as b
    I = 64
    g = (2.0 ** torch.linspace(5, 120, I)).bfloat16()
    h, dv = torch.ones((1, 2 * I)).bfloat16(), torch.full((1, I), 2.0).bfloat16()
    h[0, :I] = g
    dh, _ = b.expert_gated_backward(h.to(gpu), dv.to(gpu), fp8=False)
    assert torch.equal(dh[0, :I].cpu(), dv[0])
    assert torch.equal(dh[0, I:].cpu(), 2 * g)
