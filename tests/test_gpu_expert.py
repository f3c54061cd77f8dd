"""GPU tests of the expert products (moe_expert_gemm, moe_expert_gated_gemm) against a 64-bit
reference: ragged and empty experts, every edge of the tiles, both directions and output types,
rows of other experts beside NaN, strides of views, streams and graphs, offsets past 32 bits."""
import numpy as np
import pytest
import torch

import _expert_ref as ref

pytestmark = pytest.mark.gpu

COUNTS = {
    "one_row": [1],
    "one_token_of_many": [0, 0, 1, 0, 1, 0, 0, 1],
    "empty": [0, 0, 0],
    "tile_edges": [127, 128, 129, 0, 1, 255, 257],
    "small": [5, 0, 31, 33, 2, 64, 65, 0],
    "skewed": [700, 1, 0, 3, 90, 0, 0, 12],
    "full": [256, 257, 255, 511, 0, 700],
    "one_full": [385],
}


@pytest.fixture(scope="module")
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from combine_moe_route_gb300 import build
    build.build()
    return torch.device("cuda:0")


def _to(gpu, inp):
    return [inp[k].to(gpu) for k in ("a", "a_scale", "w", "w_scale", "off")]


@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("N,C", [(128, 128), (16, 16), (208, 144), (256, 640), (400, 272), (640, 128), (1328, 400)])
@pytest.mark.parametrize("name", sorted(COUNTS))
def test_product(gpu, name, N, C, transpose):
    from combine_moe_route_gb300 import binding as b
    rng = np.random.default_rng(N * 7 + C)
    inp = ref.product_inputs(COUNTS[name], N, C, rng, transpose)
    want, mag = ref.product(inp, transpose)
    bound = ref.product_bound(mag, C)
    args = _to(gpu, inp)
    o32 = b.expert_gemm(*args, transpose=transpose, out_dtype=torch.float32).cpu().double()
    o16 = b.expert_gemm(*args, transpose=transpose).cpu().double()
    assert ((o32 - want).abs() <= bound).all()
    assert ((o16 - want).abs() <= bound + 2.0 ** -8 * want.abs()).all()


@pytest.mark.parametrize("C", [2048, 7168])
@pytest.mark.parametrize("transpose", [False, True])
def test_product_long_contraction(gpu, C, transpose):
    from combine_moe_route_gb300 import binding as b
    inp = ref.product_inputs([40, 0, 130], 384, C, np.random.default_rng(C), transpose)
    want, mag = ref.product(inp, transpose)
    o = b.expert_gemm(*_to(gpu, inp), transpose=transpose, out_dtype=torch.float32).cpu().double()
    assert ((o - want).abs() <= ref.product_bound(mag, C)).all()
    # on average the sums are those of fp32: far below the worst case
    assert float((o - want).norm() / want.norm()) < 1e-6


@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("C", [512, 1040, 2048, 4112, 7168])
@pytest.mark.parametrize("counts", [[1], [3, 0, 1], [33], [70, 20], [128]])
def test_few_tiles_over_a_long_contraction(gpu, counts, C, transpose):
    """Tiles so few that blocks share a tile's channels and add up: 128 and 144 columns over short
    and long contractions, rows that spread over the blocks and rows that do not; the sums repeat
    bit for bit."""
    from combine_moe_route_gb300 import binding as b
    for N in (128, 144):
        inp = ref.product_inputs(counts, N, C, np.random.default_rng(C + N), transpose)
        want, mag = ref.product(inp, transpose)
        args = _to(gpu, inp)
        o = b.expert_gemm(*args, transpose=transpose, out_dtype=torch.float32)
        assert ((o.cpu().double() - want).abs() <= ref.product_bound(mag, C)).all()
        assert float((o.cpu().double() - want).norm() / want.norm()) < 1e-6
        o16 = b.expert_gemm(*args, transpose=transpose)
        assert torch.equal(o16, o.bfloat16())
        for _ in range(3):
            assert torch.equal(b.expert_gemm(*args, transpose=transpose, out_dtype=torch.float32), o)
    if not transpose and C % 128 == 0:
        I = 128
        inp = ref.product_inputs(counts, 2 * I, C, np.random.default_rng(C))
        p, mag = ref.product(inp)
        err = ref.product_bound(mag, C)
        g, u, eg, eu = p[:, :I], p[:, I:], err[:, :I], err[:, I:]
        v = ref.gate(g, u)
        verr = 1.1 * eg * (u.abs() + eu) + g.abs() * eu + 8 * 2.0 ** -24 * v.abs()
        r = b.expert_gated_gemm(*_to(gpu, inp), save_h=True)
        assert ref.quantized_ok(r.q.cpu(), r.scale.cpu(), v, verr) == (True, True)
        assert ((r.h.cpu().double() - p).abs() <= err + 2.0 ** -8 * p.abs()).all()


@pytest.mark.parametrize("save", [False, True])
@pytest.mark.parametrize("I,C", [(128, 128), (256, 144), (384, 640), (640, 2048)])
@pytest.mark.parametrize("name", sorted(COUNTS))
def test_gated(gpu, name, I, C, save):
    from combine_moe_route_gb300 import binding as b
    inp = ref.product_inputs(COUNTS[name], 2 * I, C, np.random.default_rng(I + C))
    p, mag = ref.product(inp)
    err = ref.product_bound(mag, C)
    g, u, eg, eu = p[:, :I], p[:, I:], err[:, :I], err[:, I:]
    v = ref.gate(g, u)
    # silu's slope is below 1.1 and silu(g) <= |g|; expf and the division add 8 roundings
    verr = 1.1 * eg * (u.abs() + eu) + g.abs() * eu + 8 * 2.0 ** -24 * v.abs()
    r = b.expert_gated_gemm(*_to(gpu, inp), save_h=save)
    if p.shape[0]:
        assert ref.quantized_ok(r.q.cpu(), r.scale.cpu(), v, verr) == (True, True)
    if save:
        assert ((r.h.cpu().double() - p).abs() <= err + 2.0 ** -8 * p.abs()).all()
    else:
        assert r.h is None


def test_extreme_gates(gpu):
    """Gates of +-1e4 and zero blocks: silu saturates without NaN, a zero block keeps a finite scale."""
    from combine_moe_route_gb300 import binding as b
    I, C = 128, 128
    a = torch.zeros((3, C))
    a[0, 0], a[1, 0] = 1.0, -1.0
    w = torch.zeros((1, 2 * I, C))
    w[0, :I, 0], w[0, I:, 0] = 448.0, 2.0
    args = [a.to(torch.float8_e4m3fn).to(gpu), torch.full((3, 1), 25.0, device=gpu),
            w.to(torch.float8_e4m3fn).to(gpu), torch.ones((1, 2, 1), device=gpu),
            torch.tensor([0, 3], dtype=torch.int32, device=gpu)]
    r = b.expert_gated_gemm(*args)
    v = r.q.float() * r.scale
    assert torch.equal(v[0].cpu(), torch.full((I,), np.float32(11200.0 * 50.0)).float())
    assert torch.equal(v[1].cpu().abs(), torch.zeros(I)) and torch.equal(v[2].cpu().abs(), torch.zeros(I))
    assert torch.isfinite(r.scale).all()


@pytest.mark.parametrize("transpose", [False, True])
def test_nan_stays_in_its_row_and_expert(gpu, transpose):
    from combine_moe_route_gb300 import binding as b
    counts, N, C = [3, 70, 2, 140], 272, 256
    rng = np.random.default_rng(3)
    inp = ref.product_inputs(counts, N, C, rng, transpose)
    clean = b.expert_gemm(*_to(gpu, inp), transpose=transpose)
    inp["a_scale"][10, 0] = float("nan")                     # a row of expert 1
    inp["w_scale"][2] = float("inf")                         # all of expert 2
    got = b.expert_gemm(*_to(gpu, inp), transpose=transpose)
    keep = [r for r in range(sum(counts)) if r != 10 and not 73 <= r < 75]
    assert torch.equal(got[keep], clean[keep])
    assert torch.isnan(got[10]).all() and not torch.isfinite(got[73:75]).any()


def test_rows_of_no_expert_are_left(gpu):
    """Offsets that cover a part of the rows: the others keep what they held."""
    from combine_moe_route_gb300 import binding as b
    inp = ref.product_inputs([10, 150, 40], 256, 128, np.random.default_rng(4))
    inp["off"] = torch.tensor([5, 5, 140, 170], dtype=torch.int32)
    want, mag = ref.product(inp)
    out = torch.full((200, 256), 7.0, device=gpu)
    b.expert_gemm(*_to(gpu, inp), out=out)
    out = out.cpu().double()
    assert (out[:5] == 7).all() and (out[170:] == 7).all()
    assert ((out[5:170] - want[5:170]).abs() <= ref.product_bound(mag, 128)[5:170]).all()
    q = torch.full((200, 128), 3.0, device=gpu).to(torch.float8_e4m3fn)
    s = torch.full((200, 1), 5.0, device=gpu)
    b.expert_gated_gemm(*_to(gpu, inp), out=q, out_scale=s)
    for lo, hi in ((0, 5), (170, 200)):
        assert (q[lo:hi].float() == 3).all() and (s[lo:hi] == 5).all()


@pytest.mark.parametrize("off", [[0, 400, 100, 300], [-50, 20, 60, 1000], [300, 200, 100, 0], [2 ** 30, 0, 5, 2 ** 31 - 1]])
def test_offsets_out_of_range_stay_inside_the_buffers(gpu, off):
    """Offsets that decrease or leave [0, rows] are clamped: nothing outside the output is written."""
    from combine_moe_route_gb300 import binding as b
    inp = ref.product_inputs([100, 100, 100], 128, 128, np.random.default_rng(5))
    inp["off"] = torch.tensor(off, dtype=torch.int32)
    big = torch.full((500, 128), 7.0, device=gpu)
    b.expert_gemm(*_to(gpu, inp), out=big[100:400])
    torch.cuda.synchronize()
    assert (big[:100] == 7).all() and (big[400:] == 7).all()


@pytest.mark.parametrize("transpose", [False, True])
def test_views_at_sixteen_bytes(gpu, transpose):
    """Tensors that start 16 bytes into an allocation, and scales at 4 bytes."""
    from combine_moe_route_gb300 import binding as b
    inp = ref.product_inputs([33, 100], 144, 208, np.random.default_rng(6), transpose)

    def shifted(t, n):
        flat = torch.empty(t.numel() + n, dtype=t.dtype, device=gpu)
        v = flat[n:].view(t.shape)
        v.copy_(t)
        return v

    args = [shifted(inp["a"], 16), shifted(inp["a_scale"], 1), shifted(inp["w"], 16), shifted(inp["w_scale"], 1),
            shifted(inp["off"], 1)]
    want = b.expert_gemm(*_to(gpu, inp), transpose=transpose)
    out = shifted(torch.zeros((133, 144), dtype=torch.bfloat16), 8)
    assert torch.equal(b.expert_gemm(*args, transpose=transpose, out=out), want)


def test_repeats_bit_for_bit_on_other_streams_and_in_graphs(gpu):
    from combine_moe_route_gb300 import binding as b
    inp = ref.product_inputs([200, 0, 129, 5], 512, 1024, np.random.default_rng(7))
    args = _to(gpu, inp)
    want = b.expert_gemm(*args)
    wq = b.expert_gated_gemm(*args, save_h=True)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    out = torch.empty_like(want)
    g2 = b.GatedResult(torch.empty_like(wq.q), torch.empty_like(wq.scale), torch.empty_like(wq.h))
    st.wait_stream(torch.cuda.current_stream())
    b.expert_gemm(*args, out=out, stream=st)
    st.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.expert_gemm(*args, out=out)
        b.expert_gated_gemm(*args, out=g2.q, out_scale=g2.scale, h=g2.h)
    for _ in range(3):
        out.zero_()
        g2.q.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        assert torch.equal(g2.q.view(torch.uint8), wq.q.view(torch.uint8))
        assert torch.equal(g2.scale, wq.scale) and torch.equal(g2.h, wq.h)


@pytest.mark.parametrize("transpose", [False, True])
def test_offsets_past_32_bits(gpu, transpose):
    """out, and a weight, of more than 2^31 elements: the last rows are right."""
    from combine_moe_route_gb300 import binding as b
    rows, N, C = 300_007, 7168, 16
    gen = torch.Generator(device=gpu).manual_seed(8)
    a = torch.randn((rows, C), generator=gen, device=gpu).to(torch.float8_e4m3fn)
    sa = torch.rand((rows, 1), generator=gen, device=gpu) + 0.5
    shape = (2, C, N) if transpose else (2, N, C)
    w = torch.randn(shape, generator=gen, device=gpu).to(torch.float8_e4m3fn)
    sw = torch.rand((2, ref.blocks(shape[1]), ref.blocks(shape[2])), generator=gen, device=gpu) + 0.5
    off = torch.tensor([0, 150_001, rows], dtype=torch.int32, device=gpu)
    out = b.expert_gemm(a, sa, w, sw, off, transpose=transpose)
    for lo, hi, e in ((0, 130, 0), (150_001, 150_130, 1), (rows - 200, rows, 1)):
        inp = dict(a=a[lo:hi].cpu(), a_scale=sa[lo:hi].cpu(), w=w[e:e + 1].cpu(), w_scale=sw[e:e + 1].cpu(),
                   off=torch.tensor([0, hi - lo]))
        want, mag = ref.product(inp, transpose)
        got = out[lo:hi].cpu().double()
        assert ((got - want).abs() <= ref.product_bound(mag, C) + 2.0 ** -8 * want.abs()).all()


def test_weight_past_32_bits(gpu):
    from combine_moe_route_gb300 import binding as b
    E, N, C = 160, 2048, 7168                                # 2.3e9 weights
    gen = torch.Generator(device=gpu).manual_seed(9)
    w = torch.empty((E, N, C), dtype=torch.float8_e4m3fn, device=gpu)
    for e in range(0, E, 16):
        w[e:e + 16] = torch.randn((16, N, C), generator=gen, device=gpu, dtype=torch.bfloat16).mul_(64).to(w.dtype)
    sw = torch.rand((E, N // 128, C // 128), generator=gen, device=gpu)
    a = torch.randn((E, C), generator=gen, device=gpu).to(torch.float8_e4m3fn)
    sa = torch.rand((E, C // 128), generator=gen, device=gpu)
    off = torch.arange(E + 1, dtype=torch.int32, device=gpu)
    out = b.expert_gemm(a, sa, w, sw, off, out_dtype=torch.float32)
    for e in (0, 80, E - 1):
        inp = dict(a=a[e:e + 1].cpu(), a_scale=sa[e:e + 1].cpu(), w=w[e:e + 1].cpu(), w_scale=sw[e:e + 1].cpu(),
                   off=torch.tensor([0, 1]))
        want, mag = ref.product(inp)
        assert ((out[e:e + 1].cpu().double() - want).abs() <= ref.product_bound(mag, C)).all()


def test_gradient_of_the_input_against_differences(gpu):
    """The transposed product is the gradient of <dout, product> by its input: central differences of
    the 64-bit forward (linear in the input, so exact up to its own rounding)."""
    from combine_moe_route_gb300 import binding as b
    counts, N, C = [4, 0, 3], 256, 144
    rng = np.random.default_rng(10)
    fwd = ref.product_inputs(counts, N, C, rng)
    d = ref.product_inputs(counts, C, N, rng, True)          # quantised dout [rows, N]
    got = b.expert_gemm(d["a"].to(gpu), d["a_scale"].to(gpu), fwd["w"].to(gpu), fwd["w_scale"].to(gpu),
                        fwd["off"].to(gpu), transpose=True, out_dtype=torch.float32).cpu().double()
    dout = d["a"].double() * d["a_scale"].double().repeat_interleave(128, 1)[:, :N]
    w = ref._dequant_weight(fwd["w"], fwd["w_scale"])
    owner = np.repeat(np.arange(3), counts)
    x = torch.from_numpy(rng.standard_normal((7, C)))

    def loss(v, r):
        return float((dout[r] * (w[owner[r]] @ v)).sum())

    d["w"], d["w_scale"] = fwd["w"], fwd["w_scale"]
    _, mag = ref.product(d, True)
    for r in range(7):
        for c in rng.integers(0, C, 12):
            h = torch.zeros(C, dtype=torch.float64)
            h[c] = 0.5
            diff = loss(x[r] + h, r) - loss(x[r] - h, r)
            assert abs(got[r, c] - diff) <= float(ref.product_bound(mag, N)[r, c]) + 1e-9 * float(mag[r].max())
