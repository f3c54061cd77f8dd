"""GPU tests of moe_rms_norm and its gradient against 64-bit references."""
import numpy as np
import pytest
import torch

import _expert_ref as eref

pytestmark = pytest.mark.gpu
EPS = 1e-6


@pytest.fixture(scope="module")
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from combine_moe_route_gb300 import build
    build.build()
    return torch.device("cuda:0")


SHAPES = [(1, 8), (3, 40), (5, 128), (259, 256), (7, 264), (130, 512), (9, 1024), (6, 1032), (33, 2048), (4, 2880),
          (17, 4096), (3, 5120), (2, 6152), (1003, 7168), (5, 8192), (3, 8200), (2, 12288), (4, 16384)]


def _rows(gpu, gen, T, H, size=1.0):
    return (torch.randn((T, H), generator=gen, device=gpu) * size).bfloat16()


def norm64(s, w, eps=EPS):
    r = 1.0 / torch.sqrt((s * s).mean(1, keepdim=True) + eps)
    return s * r * w, r


# fp32: a sum of H squares in any order is off by at most H / 32 + 32 roundings along the deepest chain
# of its tree (a thread's own terms, then the team's), relative to the sum; its root halves that; r,
# the two products and the additions before add under 8 roundings.
def rel_bound(H):
    return (H / 64 + 32) * 2.0 ** -24


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("T,H", SHAPES)
def test_norm(gpu, T, H, residual):
    from combine_moe_route_gb300 import binding as b
    gen = torch.Generator(device=gpu).manual_seed(T + H)
    x, w = _rows(gpu, gen, T, H), (1 + 0.3 * torch.randn(H, generator=gen, device=gpu)).bfloat16()
    res = _rows(gpu, gen, T, H, 3.0) if residual else None
    fp8 = H % 128 == 0
    n = b.rms_norm(x, w, residual=res, eps=EPS, fp8=fp8)
    s = x.double() + (res.double() if residual else 0)
    y, _ = norm64(s, w.double())
    err = rel_bound(H) * y.abs() + (2.0 ** -24 * (x.double().abs() + res.double().abs()) * (y / s).nan_to_num().abs()
                                    if residual else 0)
    assert ((n.y.double() - y).abs() <= err + 2.0 ** -8 * y.abs()).all()
    if residual:
        assert torch.equal(n.h, (x.float() + res.float()).bfloat16())
    else:
        assert n.h is x
    if fp8:
        assert eref.quantized_ok(n.q.cpu(), n.scale.cpu(), y.cpu(), err.cpu()) == (True, True)
    else:
        assert n.q is None and n.scale is None


def test_in_place_and_rows_alone(gpu):
    from combine_moe_route_gb300 import binding as b
    gen = torch.Generator(device=gpu).manual_seed(0)
    for H in (256, 7168):
        x, res = _rows(gpu, gen, 70, H), _rows(gpu, gen, 70, H)
        w = _rows(gpu, gen, 1, H)[0]
        n = b.rms_norm(x, w, residual=res)
        x2, res2 = x.clone(), res.clone()
        m = b.rms_norm(x2, w, residual=res2, out=x2, out_h=res2)
        assert torch.equal(m.y, n.y) and torch.equal(m.h, n.h) and m.y is x2 and m.h is res2
        for bad in (float("nan"), float("inf")):
            y = x.clone()
            y[3, 5] = bad
            got = b.rms_norm(y, w, residual=res)
            keep = torch.arange(70, device=gpu) != 3
            assert torch.equal(got.y[keep], n.y[keep]) and got.y[3].isnan().any()


def test_zero_rows_and_none(gpu):
    from combine_moe_route_gb300 import binding as b
    w = torch.ones(128, device=gpu, dtype=torch.bfloat16)
    n = b.rms_norm(torch.zeros((3, 128), device=gpu, dtype=torch.bfloat16), w, fp8=True)
    assert (n.y == 0).all() and (n.q.float() == 0).all() and torch.isfinite(n.scale).all()
    empty = torch.empty((0, 128), device=gpu, dtype=torch.bfloat16)
    assert b.rms_norm(empty, w, fp8=True).y.shape == (0, 128)
    g = b.rms_norm_backward(empty, empty, w, dweight=torch.full((128,), 3.0, device=gpu))
    assert g.dx.shape == (0, 128) and (g.dweight == 0).all()


def grad64(dy, h, w, dh, eps=EPS):
    n64, r = norm64(h, torch.ones_like(w), eps)
    g = dy * w
    return r * (g - n64 * (g * n64).mean(1, keepdim=True)) + (dh if dh is not None else 0), (dy * n64).sum(0), n64, g, r


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("T,H", SHAPES)
def test_gradient(gpu, T, H, residual):
    from combine_moe_route_gb300 import binding as b
    gen = torch.Generator(device=gpu).manual_seed(T * 3 + H)
    h, dy = _rows(gpu, gen, T, H, 3.0), _rows(gpu, gen, T, H, 1e-3)
    dh = _rows(gpu, gen, T, H, 1e-3) if residual else None
    w = (1 + 0.3 * torch.randn(H, generator=gen, device=gpu)).bfloat16()
    got = b.rms_norm_backward(dy, h, w, dh=dh, eps=EPS)
    dx, dw, n, g, r = grad64(dy.double(), h.double(), w.double(), dh.double() if residual else None)
    # the sum of g n: rel_bound of its terms' magnitudes
    err = rel_bound(H) * r * (g.abs() + 3 * n.abs() * (g * n).abs().mean(1, keepdim=True))
    err = err + 2.0 ** -8 * dx.abs() + 2.0 ** -23 * (dx.abs() + (dh.double().abs() if residual else 0))
    assert ((got.dx.double() - dx).abs() <= err).all()
    # dweight: T terms, in runs of a team's rows and then over the teams
    assert ((got.dweight.double() - dw).abs() <= (T * 2.0 ** -24 + rel_bound(H)) * (dy.double() * n).abs().sum(0)).all()
    again = b.rms_norm_backward(dy, h, w, dh=dh, eps=EPS)
    assert torch.equal(again.dx, got.dx) and torch.equal(again.dweight, got.dweight)


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("H", [1600, 2400, 3600, 4800, 5760, 7200, 9600, 14400])
def test_gradient_of_rows_that_fill_the_ring(gpu, H, residual):
    """Rows whose stages take all of the shared memory, or nearly, and more rows than blocks."""
    from combine_moe_route_gb300 import binding as b
    gen = torch.Generator(device=gpu).manual_seed(H)
    T = 700
    h, dy = _rows(gpu, gen, T, H, 3.0), _rows(gpu, gen, T, H)
    dh = _rows(gpu, gen, T, H) if residual else None
    w = _rows(gpu, gen, 1, H)[0]
    got = b.rms_norm_backward(dy, h, w, dh=dh, eps=EPS)
    dx, dw, n, g, r = grad64(dy.double(), h.double(), w.double(), dh.double() if residual else None)
    err = rel_bound(H) * r * (g.abs() + 3 * n.abs() * (g * n).abs().mean(1, keepdim=True))
    err = err + 2.0 ** -8 * dx.abs() + 2.0 ** -23 * (dx.abs() + (dh.double().abs() if residual else 0))
    assert ((got.dx.double() - dx).abs() <= err).all()
    assert ((got.dweight.double() - dw).abs() <= (T * 2.0 ** -24 + rel_bound(H)) * (dy.double() * n).abs().sum(0)).all()


def test_gradient_against_differences(gpu):
    """dx and dweight against central differences of the 64-bit norm at the kernel's own bf16 inputs."""
    from combine_moe_route_gb300 import binding as b
    gen = torch.Generator(device=gpu).manual_seed(5)
    T, H = 3, 64
    h, dy, w = _rows(gpu, gen, T, H, 2.0), _rows(gpu, gen, T, H), _rows(gpu, gen, 1, H)[0]
    got = b.rms_norm_backward(dy, h, w, eps=1e-3)

    def loss(h64, w64):
        return (norm64(h64, w64, 1e-3)[0] * dy.double()).sum()

    step = 1e-6
    for i, j in ((0, 0), (1, 7), (2, 63)):
        e = torch.zeros((T, H), dtype=torch.float64, device=gpu)
        e[i, j] = step
        d = (loss(h.double() + e, w.double()) - loss(h.double() - e, w.double())) / (2 * step)
        # 64-bit differences: third derivatives of order 1 times step^2, and 2^-52 of a loss of about 100 over step
        assert abs(got.dx[i, j].double() - d) <= 2.0 ** -8 * abs(d) + 1e-6
        d = (loss(h.double(), w.double() + e[i]) - loss(h.double(), w.double() - e[i])) / (2 * step)
        assert abs(got.dweight[j].double() - d) <= 2.0 ** -18 * (dy.double() * h.double()).abs().sum() / H + 1e-6


def test_gradient_in_place_workspace_and_graph(gpu):
    from combine_moe_route_gb300 import binding as b
    gen = torch.Generator(device=gpu).manual_seed(6)
    for T, H in ((700, 256), (600, 4096)):
        h, dy, dh = (_rows(gpu, gen, T, H) for _ in range(3))
        w = _rows(gpu, gen, 1, H)[0]
        want = b.rms_norm_backward(dy, h, w, dh=dh)
        for name in ("dy", "h", "dh"):
            t = dict(dy=dy.clone(), h=h.clone(), dh=dh.clone())
            got = b.rms_norm_backward(t["dy"], t["h"], w, dh=t["dh"], out=t[name])
            assert torch.equal(got.dx, want.dx) and torch.equal(got.dweight, want.dweight) and got.dx is t[name]
        ws = torch.full((b.rms_norm_workspace_bytes(T, H),), 255, dtype=torch.uint8, device=gpu)   # NaN before
        got = b.rms_norm_backward(dy, h, w, dh=dh, workspace=ws)
        assert torch.equal(got.dweight, want.dweight)
        with pytest.raises(b.MoeError):
            b.rms_norm_backward(dy, h, w, workspace=ws[:-16])
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        got = b.rms_norm_backward(dy, h, w, dh=dh, stream=side)
        side.synchronize()
        assert torch.equal(got.dx, want.dx) and torch.equal(got.dweight, want.dweight)
        torch.cuda.synchronize()
        graphs, outs = [], []
        for _ in range(2):   # two graphs, a workspace each
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                outs.append(b.rms_norm_backward(dy, h, w, dh=dh))
            graphs.append(graph)
        dy.copy_(_rows(gpu, gen, T, H))
        for graph in graphs:
            graph.replay()
        want = b.rms_norm_backward(dy, h, w, dh=dh)
        for o in outs:
            assert torch.equal(o.dx, want.dx) and torch.equal(o.dweight, want.dweight)
