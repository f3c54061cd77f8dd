"""GPU tests of the gradients of the combine, the dispatch scatter, the router's softmax and the
gate, against 64-bit formulas and against differences of the 64-bit forward."""
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


def _inputs(T, K, H, E, seed, rows=None, dropped=0.0):
    rng = np.random.default_rng(seed)
    rows = T * K if rows is None else rows
    at = rng.permutation(max(rows, T * K))[:T * K].astype(np.int32)
    at[rng.random(T * K) < dropped] = -1
    at[at >= rows] = rows + 5
    logits = torch.from_numpy(rng.standard_normal((T, E)))
    top, idx = torch.topk(logits, K, dim=1)
    return dict(dout=torch.from_numpy(rng.standard_normal((T, H)).astype(np.float32)).bfloat16(),
                y=torch.from_numpy(rng.standard_normal((rows, H)).astype(np.float32)).bfloat16(),
                tok2row=torch.from_numpy(at), w=torch.softmax(top, 1).float(), idx=idx.int(), logits=logits, E=E)


SHAPES = [(1, 1, 8, 1), (1, 8, 7168, 256), (3, 2, 264, 16), (259, 2, 256, 16), (37, 8, 1032, 384), (5, 9, 128, 60),
          (11, 32, 640, 1024), (64, 6, 2048, 64)]


@pytest.mark.parametrize("dropped", [0.0, 0.3])
@pytest.mark.parametrize("T,K,H,E", SHAPES)
def test_combine_backward(gpu, T, K, H, E, dropped):
    from combine_moe_route_gb300 import binding as b
    i = _inputs(T, K, H, E, T + K + H, rows=T * K + 7, dropped=dropped)
    dy, dw, dl, dw_err, dl_err = ref.combine_grads(i["dout"], i["y"], i["tok2row"], i["w"], i["idx"], E)
    out = torch.full((T * K + 7, H), 7.0, dtype=torch.bfloat16, device=gpu)
    r = b.combine_backward(i["dout"].to(gpu), i["y"].to(gpu), i["tok2row"].to(gpu), i["w"].to(gpu),
                           topk_idx=i["idx"].to(gpu), E=E, out=out)
    got = r.dy.cpu()
    free = torch.isnan(dy[:, 0])
    assert (got[free] == 7).all()
    # a product of a fp32 weight and a bf16 value, rounded to fp32 and then to bf16: as computed here
    at = i["tok2row"].long().view(T, K)
    for j in range(K):
        ok = (at[:, j] >= 0) & (at[:, j] < T * K + 7)
        want = (i["w"][:, j:j + 1] * i["dout"].float()).bfloat16()
        assert torch.equal(got[at[ok, j]], want[ok])
    assert ((r.dtopk_w.cpu().double() - dw).abs() <= dw_err).all()
    assert ((r.dlogits.cpu().double() - dl).abs() <= dl_err).all()
    only = b.combine_backward(i["dout"].to(gpu), i["y"].to(gpu), i["tok2row"].to(gpu), i["w"].to(gpu))
    assert only.dlogits is None and torch.equal(only.dtopk_w, r.dtopk_w)


@pytest.mark.parametrize("dropped", [0.0, 0.3])
@pytest.mark.parametrize("T,K,H,E", [s for s in SHAPES if s[2] % 128 == 0])
def test_combine_backward_quantised(gpu, T, K, H, E, dropped):
    """Codes and scales equal the dispatch's rule applied in fp32, bit for bit."""
    from combine_moe_route_gb300 import binding as b
    i = _inputs(T, K, H, E, T + K + H + 1, dropped=dropped)
    i["dout"][0, :min(H, 256)] = 0                                    # zero blocks
    i["w"][T // 2] *= 2.0 ** -100
    q = torch.full((T * K, H), 7.0, device=gpu).to(torch.float8_e4m3fn)
    s = torch.full((T * K, H // 128), 5.0, device=gpu)
    r = b.combine_backward(i["dout"].to(gpu), i["y"].to(gpu), i["tok2row"].to(gpu), i["w"].to(gpu), fp8=True, out=q,
                           out_scale=s)
    at = i["tok2row"].long().view(T, K)
    written = torch.zeros(T * K, dtype=torch.bool)
    gq, gs = r.dy.cpu().view(torch.uint8), r.dy_scale.cpu()
    for j in range(K):
        ok = (at[:, j] >= 0) & (at[:, j] < T * K)
        wq, ws = ref.quantize_f32(i["w"][:, j:j + 1] * i["dout"].float())
        wq = wq.view(torch.uint8)
        same = (gq[at[ok, j]] == wq[ok]) | ((gq[at[ok, j]] | wq[ok]) == 0x80)   # +0 and -0 are both zero
        assert same.all()
        assert torch.equal(gs[at[ok, j]], ws[ok])
        written[at[ok, j]] = True
    assert (r.dy.cpu().float()[~written] == 7).all() and (gs[~written] == 5).all()
    _, dw, _, dw_err, _ = ref.combine_grads(i["dout"], i["y"], i["tok2row"], i["w"], i["idx"], E)
    assert ((r.dtopk_w.cpu().double() - dw).abs() <= dw_err).all()


def test_combine_backward_without_rows(gpu):
    """A buffer of no rows: every weight's gradient is zero and nothing else is written."""
    from combine_moe_route_gb300 import binding as b
    i = _inputs(9, 3, 256, 8, 0, rows=0)
    r = b.combine_backward(i["dout"].to(gpu), i["y"].to(gpu), i["tok2row"].to(gpu), i["w"].to(gpu),
                           topk_idx=i["idx"].to(gpu), E=8)
    assert (r.dtopk_w == 0).all() and (r.dlogits == 0).all()
    assert b.combine_backward(i["dout"][:0].to(gpu), i["y"].to(gpu), i["tok2row"][:0].to(gpu),
                              i["w"][:0].to(gpu)).dtopk_w.shape == (0, 3)


def test_combine_backward_identity_map_and_nan(gpu):
    from combine_moe_route_gb300 import binding as b
    i = _inputs(6, 4, 384, 16, 1)
    ident = torch.arange(24, dtype=torch.int32)
    y = i["y"].clone()
    y[4, 7] = float("nan")                                            # token 1, copy 0
    y[9, 0] = float("inf")                                            # token 2, copy 1
    args = (i["dout"].to(gpu), y.to(gpu))
    r0 = b.combine_backward(*args, None, i["w"].to(gpu), topk_idx=i["idx"].to(gpu), E=16)
    r1 = b.combine_backward(*args, ident.to(gpu), i["w"].to(gpu), topk_idx=i["idx"].to(gpu), E=16)
    assert torch.equal(r0.dy, r1.dy)
    bad = torch.zeros((6, 4), dtype=torch.bool)
    bad[1, 0] = bad[2, 1] = True
    assert torch.equal(~torch.isfinite(r0.dtopk_w.cpu()), bad)
    assert torch.isfinite(r0.dlogits[[0, 3, 4, 5]]).all()
    assert torch.isfinite(r0.dy.float()).all()


@pytest.mark.parametrize("T,K,H,E", SHAPES)
@pytest.mark.parametrize("dropped", [0.0, 0.3])
def test_dispatch_backward(gpu, T, K, H, E, dropped):
    from combine_moe_route_gb300 import binding as b
    i = _inputs(T, K, H, E, T * K + H, rows=T * K + 3, dropped=dropped)
    rows = i["y"]
    at = i["tok2row"].long().view(T, K)
    ok = (at >= 0) & (at < T * K + 3)
    want = torch.zeros((T, H))
    for j in range(K):                                                # fp32, ascending j: bit for bit
        want += rows.float()[at[:, j].clamp(0, T * K + 2)] * ok[:, j:j + 1]
    o32 = b.dispatch_backward(rows.to(gpu), i["tok2row"].to(gpu), K, out_dtype=torch.float32)
    o16 = b.dispatch_backward(rows.to(gpu), i["tok2row"].to(gpu), K)
    assert torch.equal(o32.cpu(), want)
    assert torch.equal(o16.cpu(), want.bfloat16())


@pytest.mark.parametrize("layout", ["ragged", "low_latency"])
def test_gradients_through_both_layouts_against_differences(gpu, layout):
    """combine(w, dispatch(x)) in each layout: the gradients equal central differences of the
    64-bit forward by the tokens, the expert outputs and the logits."""
    from combine_moe_route_gb300 import binding as b
    B, E, K, H, C = [5, 0, 9, 2], 8, 3, 256, 9
    T = sum(B)
    rng = np.random.default_rng(12)
    x = torch.from_numpy(rng.standard_normal((T, H)).astype(np.float32)).bfloat16()
    logits = torch.from_numpy(rng.standard_normal((T, E)).astype(np.float32))
    dout = torch.from_numpy(rng.standard_normal((T, H)).astype(np.float32)).bfloat16()
    idx, w = b.route_topk(logits.to(gpu), K)
    if layout == "ragged":
        d = b.dispatch(x.to(gpu), idx, B, E)
        rows = T * K
    else:
        d = b.dispatch_ll(x.to(gpu), idx, B, E, C)
        rows = E * len(B) * C
    y = torch.from_numpy(rng.standard_normal((rows, H)).astype(np.float32)).bfloat16()
    r = b.combine_backward(dout.to(gpu), y.to(gpu), d.tok2row, w, topk_idx=idx, E=E)
    at, ids = d.tok2row.long().cpu().view(T, K), idx.long().cpu()

    def loss(lg, yy):
        p = torch.softmax(lg.gather(1, ids), 1)
        return float((dout.double() * (p[:, :, None] * yy[at]).sum(1)).sum())

    l64, y64 = logits.double(), y.double()
    for _ in range(20):
        t, e = int(rng.integers(T)), int(rng.integers(E))
        h = torch.zeros_like(l64)
        h[t, e] = 1e-4
        diff = (loss(l64 + h, y64) - loss(l64 - h, y64)) / 2e-4
        # fp32 sums of 256 unit normals' products, and a second-order term of 1e-8
        assert abs(float(r.dlogits[t, e]) - diff) <= 256 * 2.0 ** -24 * 256 + 1e-5
        j, c = int(rng.integers(K)), int(rng.integers(H))
        h = torch.zeros_like(y64)
        h[at[t, j], c] = 0.5
        diff = loss(l64, y64 + h) - loss(l64, y64 - h)
        assert abs(float(r.dy[at[t, j], c]) - diff) <= 2.0 ** -8 * abs(diff) + 1e-6
    drows = y.to(gpu)
    dx = b.dispatch_backward(drows, d.tok2row, K, out_dtype=torch.float32).cpu().double()

    def scatter_loss(xx):
        recv = torch.zeros((rows, H), dtype=torch.float64)
        recv[at.view(-1)] = xx.repeat_interleave(K, 0)
        return float((recv[at.view(-1)] * y64[at.view(-1)]).sum())

    for _ in range(10):
        t, c = int(rng.integers(T)), int(rng.integers(H))
        h = torch.zeros((T, H), dtype=torch.float64)
        h[t, c] = 0.5
        diff = scatter_loss(x.double() + h) - scatter_loss(x.double() - h)
        assert abs(dx[t, c] - diff) <= 1e-5


@pytest.mark.parametrize("rows,I", [(1, 8), (1, 128), (3, 24), (7, 640), (129, 2048), (1000, 136), (33, 1408)])
def test_gated_backward(gpu, rows, I):
    from combine_moe_route_gb300 import binding as b
    rng = np.random.default_rng(rows + I)
    h = torch.from_numpy(rng.standard_normal((rows, 2 * I)).astype(np.float32) * 4).bfloat16()
    dv = torch.from_numpy(rng.standard_normal((rows, I)).astype(np.float32)).bfloat16()
    h[0, :4] = torch.tensor([0.0, 200.0, -200.0, -0.0])
    g, u = h[:, :I].double(), h[:, I:].double()
    dg, du, bound = ref.gate_grad(g, u, dv.double())
    want, err = torch.cat([dg, du], 1), torch.cat([bound, bound], 1)
    o, none = b.expert_gated_backward(h.to(gpu), dv.to(gpu), fp8=False)
    assert none is None
    assert ((o.cpu().double() - want).abs() <= err + 2.0 ** -8 * want.abs() + 2.0 ** -133).all()
    if I % 128 == 0:
        q, s = b.expert_gated_backward(h.to(gpu), dv.to(gpu))
        assert ref.quantized_ok(q.cpu(), s.cpu(), want, err) == (True, True)


def test_gated_backward_against_differences(gpu):
    from combine_moe_route_gb300 import binding as b
    rng = np.random.default_rng(13)
    I = 64
    h = torch.from_numpy(rng.standard_normal((4, 2 * I)).astype(np.float32) * 2).bfloat16()
    dv = torch.from_numpy(rng.standard_normal((4, I)).astype(np.float32)).bfloat16()
    got = b.expert_gated_backward(h.to(gpu), dv.to(gpu), fp8=False)[0].cpu().double()
    step = 1e-4
    for i in range(2 * I):
        e = torch.zeros((4, 2 * I), dtype=torch.float64)
        e[:, i] = step
        lo, hi = h.double() - e, h.double() + e
        diff = ((ref.gate(hi[:, :I], hi[:, I:]) - ref.gate(lo[:, :I], lo[:, I:])) * dv.double()).sum(1) / (2 * step)
        assert ((got[:, i] - diff).abs() <= 2.0 ** -8 * diff.abs() + 1e-6).all()


def test_gated_backward_nan_and_infinite_gates(gpu):
    """A NaN reaches its own element (and its code), an infinite gate only its own."""
    from combine_moe_route_gb300 import binding as b
    I = 256
    h = torch.ones((2, 2 * I)).bfloat16()
    dv = torch.ones((2, I)).bfloat16()
    h[0, 3], h[1, 5] = float("nan"), float("-inf")
    o, _ = b.expert_gated_backward(h.to(gpu), dv.to(gpu), fp8=False)
    bad = ~torch.isfinite(o.cpu().float())
    want = torch.zeros_like(bad)
    want[0, 3] = want[0, I + 3] = want[1, 5] = want[1, I + 5] = True
    assert not (bad & ~want).any() and bad[0, 3] and bad[0, I + 3]
    q, s = b.expert_gated_backward(h.to(gpu), dv.to(gpu))
    assert torch.isfinite(s[0]).all() and torch.isnan(q.float()[0, 3]) and not torch.isnan(q.float()[0, 4:128]).any()


def test_gradients_past_32_bits(gpu):
    """Rows whose offsets pass 2^31 elements: the last ones are right."""
    from combine_moe_route_gb300 import binding as b
    T, K, H = 300_011, 1, 7168
    gen = torch.Generator(device=gpu).manual_seed(2)
    rows = torch.randn((T, H), generator=gen, device=gpu, dtype=torch.bfloat16)
    dout = torch.randn((T, H), generator=gen, device=gpu, dtype=torch.bfloat16)
    at = torch.arange(T - 1, -1, -1, dtype=torch.int32, device=gpu)
    w = torch.rand((T, K), generator=gen, device=gpu)
    r = b.combine_backward(dout, rows, at, w)
    dx = b.dispatch_backward(rows, at, K)
    for t in (0, 5, T // 2, T - 1):
        assert torch.equal(dx[t], rows[T - 1 - t])
        assert torch.equal(r.dy[T - 1 - t], (w[t] * dout[t].float()).bfloat16())
        dot = (dout[t].double() * rows[T - 1 - t].double())
        assert abs(float(r.dtopk_w[t, 0]) - float(dot.sum())) <= H * 2.0 ** -24 * float(dot.abs().sum())
    dh, _ = b.expert_gated_backward(rows, dout[:, :H // 2].contiguous(), fp8=False)
    g, u = rows[-1, :H // 2].double(), rows[-1, H // 2:].double()
    dg, du, bound = ref.gate_grad(g, u, dout[-1, :H // 2].double())
    want, err = torch.cat([dg, du]), torch.cat([bound, bound])
    assert ((dh[-1].double() - want).abs() <= err + 2.0 ** -8 * want.abs()).all()


def test_gradients_repeat_on_other_streams_and_in_graphs(gpu):
    from combine_moe_route_gb300 import binding as b
    i = _inputs(77, 8, 2048, 64, 4)
    args = [i[k].to(gpu) for k in ("dout", "y", "tok2row", "w")]
    idx = i["idx"].to(gpu)
    want = b.combine_backward(*args, topk_idx=idx, E=64, fp8=True)
    dx = b.dispatch_backward(args[1], args[2], 8)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got = b.CombineGrad(*[torch.empty_like(t) for t in (want.dy, want.dy_scale, want.dtopk_w, want.dlogits)])
    st.wait_stream(torch.cuda.current_stream())

    def again(stream=None):
        b.combine_backward(*args, topk_idx=idx, E=64, fp8=True, out=got.dy, out_scale=got.dy_scale,
                           dtopk_w=got.dtopk_w, dlogits=got.dlogits, stream=stream)

    def same():
        return (torch.equal(got.dy.view(torch.uint8), want.dy.view(torch.uint8)) and
                torch.equal(got.dy_scale, want.dy_scale) and torch.equal(got.dtopk_w, want.dtopk_w) and
                torch.equal(got.dlogits, want.dlogits))

    again(st)
    st.synchronize()
    assert same()
    out = torch.empty_like(dx)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        again()
        b.dispatch_backward(args[1], args[2], 8, out=out)
    for _ in range(2):
        got.dtopk_w.zero_()
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert same() and torch.equal(out, dx)
