"""GPU tests of the 4-bit rows (moe_quantize_mx4, moe_dequantize_mx4) and their products
(moe_expert_gemm_mx4, moe_expert_gated_gemm_mx4) against 64-bit references: codes and scales bit for
bit, every edge of the tiles, ragged and empty experts, scales at every alignment, rows beside NaN,
streams and graphs."""
import numpy as np
import pytest
import torch

import _expert_ref as eref
import _mx4_ref as ref

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


def _check_quantized(b, x, gpu):
    codes, byte = ref.quantize(x.double())
    q, s = b.quantize_mx4(x.to(gpu))
    assert torch.equal(s.cpu(), byte)
    assert torch.equal(ref.unpack(q.cpu()), codes)
    back = b.dequantize_mx4(q, s).cpu().double()
    want = ref.values(ref.pack(codes), byte)
    assert torch.equal(torch.isnan(back), torch.isnan(want))
    assert torch.equal(back.nan_to_num(), want.nan_to_num())
    v = b.dequantize_mx4(q, None)
    assert v.dtype == torch.float8_e4m3fn and torch.equal(v.cpu().double(), ref.code_values(codes))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape", [(1, 32), (3, 96), (127, 160), (1, 7168), (33, 2048), (2, 5, 2880), (64,), (4096, 32)])
def test_quantize(gpu, shape, dtype):
    from combine_moe_route_gb300 import binding as b
    rng = np.random.default_rng(sum(shape))
    x = torch.from_numpy(rng.standard_normal(shape).astype(np.float32) * np.exp2(rng.integers(-8, 8, shape)).astype(np.float32))
    _check_quantized(b, x.to(dtype), gpu)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_quantize_edges(gpu, dtype):
    """Ties, zeros of both signs, subnormals, the ends of the exponents, infinities and NaN."""
    from combine_moe_route_gb300 import binding as b
    inf = float("inf")
    ties = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0, 4.0, 6.0, 0.2490234375, 0.251953125, 7.96875, 0.0, -0.0, 1.0])
    rows = [torch.cat([ties, -ties]) * 2.0 ** k for k in (0, -3, 60, -120, -125, -127, 120)]
    rows += [torch.zeros(32), -torch.zeros(32), torch.full((32,), 2.0 ** -126), torch.full((32,), 2.0 ** -133),
             torch.full((32,), 3.3e38), torch.arange(32) * 2.0 ** -133]
    for v in (inf, -inf, float("nan")):
        r = torch.ones(32)
        r[7] = v
        rows.append(r)
    x = torch.stack(rows).to(dtype)
    _check_quantized(b, x, gpu)
    if dtype is torch.float32:
        _check_quantized(b, torch.full((2, 32), 2.0 ** -149), gpu)
        up = torch.tensor([2.0, 4.0, 2.0 ** -100]) * (1 - 2.0 ** -24)   # just under a power of two
        _check_quantized(b, up[:, None].repeat(1, 32).contiguous(), gpu)


def test_every_code_and_scale_reads_back(gpu):
    from combine_moe_route_gb300 import binding as b
    q = torch.arange(256, dtype=torch.uint8)[None].repeat(256, 1)          # [256, 256]: C = 512
    s = torch.arange(256, dtype=torch.uint8)[:, None].repeat(1, 16)
    got = b.dequantize_mx4(q.to(gpu), s.to(gpu)).cpu()
    want = ref.values(q, s).to(torch.bfloat16)
    assert torch.equal(got.isnan(), want.isnan()) and torch.equal(got.nan_to_num(), want.nan_to_num())


@pytest.mark.parametrize("N,C", [(128, 256), (16, 32), (208, 160), (256, 640), (400, 288), (640, 128), (1328, 416), (256, 1024)])
@pytest.mark.parametrize("name", sorted(COUNTS))
def test_product(gpu, name, N, C):
    from combine_moe_route_gb300 import binding as b
    inp = ref.product_inputs(COUNTS[name], N, C, np.random.default_rng(N * 7 + C))
    want, mag = ref.product(inp)
    bound = ref.product_bound(mag, C)
    args = _to(gpu, inp)
    o32 = b.expert_gemm_mx4(*args, out_dtype=torch.float32).cpu().double()
    o16 = b.expert_gemm_mx4(*args).cpu().double()
    assert ((o32 - want).abs() <= bound).all()
    assert ((o16 - want).abs() <= bound + 2.0 ** -8 * want.abs()).all()


@pytest.mark.parametrize("C", [2048, 2880, 7168])
@pytest.mark.parametrize("counts", [[1], [3, 0, 1], [33], [70, 20], [40, 0, 130], [300, 2]])
def test_long_contraction(gpu, counts, C):
    """Also tiles so few that blocks share a tile's channels; the sums repeat bit for bit."""
    from combine_moe_route_gb300 import binding as b
    for N in (128, 144, 384):
        inp = ref.product_inputs(counts, N, C, np.random.default_rng(C + N))
        want, mag = ref.product(inp)
        args = _to(gpu, inp)
        o = b.expert_gemm_mx4(*args, out_dtype=torch.float32)
        assert ((o.cpu().double() - want).abs() <= ref.product_bound(mag, C)).all()
        # on average the sums are those of fp32: far below the worst case
        assert float((o.cpu().double() - want).norm() / want.norm()) < 1e-6
        for _ in range(3):
            assert torch.equal(b.expert_gemm_mx4(*args, out_dtype=torch.float32), o)


MANY = {"pairs": [1600], "pairs_and_rests": [2000, 5, 300, 1100], "half_a_pair": [900, 770], "blocks": [700, 690, 710]}


@pytest.mark.parametrize("N,C", [(208, 160), (400, 640), (1328, 2048), (4096, 2880)])
@pytest.mark.parametrize("name", sorted(MANY))
def test_many_rows(gpu, name, N, C):
    """Pairs of blocks with and without a rest, blocks of several tiles, rings that wrap often."""
    from combine_moe_route_gb300 import binding as b
    inp = ref.product_inputs(MANY[name], N, C, np.random.default_rng(N + C))
    args = _to(gpu, inp)
    w64, a64 = ref.values(inp["w"], inp["w_scale"]), ref.values(inp["a"], inp["a_scale"])
    off = inp["off"].tolist()
    o32 = b.expert_gemm_mx4(*args, out_dtype=torch.float32)
    o16 = b.expert_gemm_mx4(*args)
    assert torch.equal(o16, o32.bfloat16())
    assert torch.equal(b.expert_gemm_mx4(*args, out_dtype=torch.float32), o32)
    for e in range(len(MANY[name])):
        rows = slice(off[e], off[e + 1])
        want, mag = a64[rows] @ w64[e].T, a64[rows].abs() @ w64[e].abs().T
        assert ((o32[rows].cpu().double() - want).abs() <= ref.product_bound(mag, C)).all()
    assert b.get_expert_error()[0] == 0


@pytest.mark.parametrize("I,C", [(96, 160), (256, 2048), (1024, 2880)])
@pytest.mark.parametrize("name", sorted(MANY))
def test_gated_many_rows(gpu, name, I, C):
    from combine_moe_route_gb300 import binding as b
    inp = ref.product_inputs(MANY[name], 2 * I, C, np.random.default_rng(I + C), spread=1)
    inp["w_scale"] -= 5
    p, mag = ref.product(inp)
    err = ref.product_bound(mag, C)
    g, u, eg, eu = p[:, :I], p[:, I:], err[:, :I], err[:, I:]
    v = eref.gate(g, u)
    bound = 1.1 * eg * (u.abs() + eu) + (g.abs() + eg) * eu + 16 * 2.0 ** -24 * v.abs()
    r = b.expert_gated_gemm_mx4(*_to(gpu, inp))
    assert ref.quantized_ok(r.q.cpu(), r.scale.cpu(), v, bound) == (True, True)


def test_result_past_32_bits(gpu):
    """70000 x 32768 values: the last rows' places are past 2^31 elements."""
    from combine_moe_route_gb300 import binding as b
    gen = torch.Generator(device=gpu).manual_seed(7)
    R, N, C = 70000, 32768, 64
    a, sa = b.quantize_mx4(torch.randn((R, C), generator=gen, device=gpu))
    w, sw = b.quantize_mx4(torch.randn((1, N, C), generator=gen, device=gpu))
    out = b.expert_gemm_mx4(a, sa, w, sw, torch.tensor([0, R], dtype=torch.int32, device=gpu))
    for rows in (slice(0, 3), slice(65530, 65545), slice(R - 70, R)):
        n = rows.stop - rows.start
        small = b.expert_gemm_mx4(a[rows].clone(), sa[rows].clone(), w, sw, torch.tensor([0, n], dtype=torch.int32, device=gpu))
        want = b.dequantize_mx4(a[rows].clone(), sa[rows].clone()).float() @ b.dequantize_mx4(w, sw)[0].float().T
        assert torch.equal(out[rows], small) and (out[rows].float() - want).abs().max() <= 2.0 ** -8 * want.abs().max()


def test_two_streams_at_once(gpu):
    from combine_moe_route_gb300 import binding as b
    gen = torch.Generator(device=gpu).manual_seed(8)
    streams, work = [torch.cuda.Stream() for _ in range(2)], []
    for i, rows in enumerate((900, 40)):
        a, sa = b.quantize_mx4(torch.randn((rows, 2048), generator=gen, device=gpu))
        w, sw = b.quantize_mx4(torch.randn((2, 512, 2048), generator=gen, device=gpu))
        off = torch.tensor([0, rows // 3, rows], dtype=torch.int32, device=gpu)
        work.append((a, sa, w, sw, off))
    want = [b.expert_gemm_mx4(*x) for x in work]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(b.expert_gemm_mx4(*work[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(g, want[i]) for g in got[i])


def test_first_call_of_a_process_inside_a_capture(gpu):
    import os
    import subprocess
    import sys
    code = """
import torch
from combine_moe_route_gb300 import binding as b
x = torch.ones((300, 512), device="cuda", dtype=torch.bfloat16)
w = torch.ones((1, 256, 512), device="cuda", dtype=torch.bfloat16)
g = torch.ones(512, device="cuda", dtype=torch.bfloat16)
off = torch.tensor([0, 300], dtype=torch.int32, device="cuda")
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    q, s = b.quantize_mx4(b.rms_norm(x, g).y)
    wq, ws = b.quantize_mx4(w)
    out = b.expert_gemm_mx4(q, s, wq, ws, off)
    grad = b.rms_norm_backward(x.repeat(1, 4), x.repeat(1, 4), g.repeat(4))
graph.replay()
torch.cuda.synchronize()
assert (out == 512).all(), out
assert torch.isfinite(grad.dweight).all()
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=110)
    assert r.returncode == 0, r.stderr[-2000:]


@pytest.mark.parametrize("I,C", [(128, 256), (32, 32), (96, 160), (256, 640), (416, 288), (160, 2048), (128, 7168)])
@pytest.mark.parametrize("name", sorted(COUNTS))
def test_gated(gpu, name, I, C):
    from combine_moe_route_gb300 import binding as b
    inp = ref.product_inputs(COUNTS[name], 2 * I, C, np.random.default_rng(I * 5 + C), spread=1)
    inp["w_scale"] -= 4   # gates of a few units
    p, mag = ref.product(inp)
    err = ref.product_bound(mag, C)
    g, u, eg, eu = p[:, :I], p[:, I:], err[:, :I], err[:, I:]
    v = eref.gate(g, u)
    # |d silu| <= 1.1, |silu| <= |g|; the gate's own roundings: under 16 of 2^-24
    bound = 1.1 * eg * (u.abs() + eu) + (g.abs() + eg) * eu + 16 * 2.0 ** -24 * v.abs()
    r = b.expert_gated_gemm_mx4(*_to(gpu, inp))
    assert r.h is None
    assert ref.quantized_ok(r.q.cpu(), r.scale.cpu(), v, bound) == (True, True)


@pytest.mark.parametrize("shift", [1, 4, 8, 16])
@pytest.mark.parametrize("C", [512, 640, 160])
def test_scales_at_every_alignment(gpu, shift, C):
    from combine_moe_route_gb300 import binding as b
    inp = ref.product_inputs([130, 3, 7], 272, C, np.random.default_rng(C))
    a, sa, w, sw, off = _to(gpu, inp)
    want = b.expert_gemm_mx4(a, sa, w, sw, off)

    def moved(s):
        room = torch.full((s.numel() + 64,), 255, dtype=torch.uint8, device=gpu)   # NaN around it
        room[shift:shift + s.numel()] = s.flatten()
        return room[shift:shift + s.numel()].view(s.shape)

    assert torch.equal(b.expert_gemm_mx4(a, moved(sa), w, sw, off), want)
    assert torch.equal(b.expert_gemm_mx4(a, sa, w, moved(sw), off), want)


@pytest.mark.parametrize("rows", [[1], [200, 33]])
def test_result_at_16_bytes(gpu, rows):
    """A result that starts between two 32-byte sectors, whole and in parts."""
    from combine_moe_route_gb300 import binding as b
    inp = ref.product_inputs(rows, 272, 2048, np.random.default_rng(9))
    args = _to(gpu, inp)
    want = b.expert_gemm_mx4(*args)
    R = want.shape[0]
    room = torch.full((R * 272 + 64,), 7.0, dtype=torch.bfloat16, device=gpu)
    out = room[8:8 + R * 272].view(R, 272)
    b.expert_gemm_mx4(*args, out=out)
    assert torch.equal(out, want) and (room[:8] == 7).all() and (room[8 + R * 272:] == 7).all()


def test_rows_stand_alone(gpu):
    """A NaN scale reaches its own row (or column) and nothing else; rows of no expert stay."""
    from combine_moe_route_gb300 import binding as b
    inp = ref.product_inputs([130, 140], 256, 512, np.random.default_rng(3))
    a, sa, w, sw, off = _to(gpu, inp)
    want = b.expert_gemm_mx4(a, sa, w, sw, off)
    sa2 = sa.clone()
    sa2[5, 3] = 255
    sa2[130] = 255
    got = b.expert_gemm_mx4(a, sa2, w, sw, off)
    keep = torch.ones(270, dtype=torch.bool, device=gpu)
    keep[5] = keep[130] = False
    assert got[5].isnan().all() and got[130].isnan().all() and torch.equal(got[keep], want[keep])
    sw2 = sw.clone()
    sw2[1, 17, 0] = 255
    got = b.expert_gemm_mx4(a, sa, w, sw2, off)
    assert got[130:, 17].isnan().all() and torch.equal(got[:130], want[:130])
    keep = torch.ones(256, dtype=torch.bool, device=gpu)
    keep[17] = False
    assert torch.equal(got[130:][:, keep], want[130:][:, keep])
    # offsets that leave rows out, and offsets out of range
    out = torch.full_like(want, 7.0)
    b.expert_gemm_mx4(a, sa, w, sw, torch.tensor([10, 130, 200], dtype=torch.int32, device=gpu), out=out)
    assert torch.equal(out[10:200], want[10:200]) and (out[:10] == 7).all() and (out[200:] == 7).all()
    out = torch.full_like(want, 7.0)
    b.expert_gemm_mx4(a, sa, w, sw, torch.tensor([-5, 130, 1 << 30], dtype=torch.int32, device=gpu), out=out)
    assert torch.equal(out, want)


def test_gated_row_with_nan(gpu):
    from combine_moe_route_gb300 import binding as b
    inp = ref.product_inputs([40], 128, 256, np.random.default_rng(4), spread=1)
    a, sa, w, sw, off = _to(gpu, inp)
    r = b.expert_gated_gemm_mx4(a, sa, w, sw, off)
    sa[3] = 255
    got = b.expert_gated_gemm_mx4(a, sa, w, sw, off)
    assert (got.scale[3] == 255).all() and (got.q[3] == 0).all()
    keep = torch.arange(40, device=gpu) != 3
    assert torch.equal(got.q[keep], r.q[keep]) and torch.equal(got.scale[keep], r.scale[keep])
    assert b.dequantize_mx4(got.q, got.scale)[3].isnan().all()


def test_scales_at_their_ends(gpu):
    """Products of scales from 2^-126 to 2^120: powers of two move the result and lose nothing."""
    from combine_moe_route_gb300 import binding as b
    inp = ref.product_inputs([20, 5], 64, 256, np.random.default_rng(5), spread=0)
    a, sa, w, sw, off = _to(gpu, inp)
    base = b.expert_gemm_mx4(a, sa, w, sw, off, out_dtype=torch.float32)
    for ka, kw in ((100, 10), (-60, -50), (127, -127), (-127, 127), (-20, 125)):
        got = b.expert_gemm_mx4(a, (sa.int() + ka).to(torch.uint8), w, (sw.int() + kw).to(torch.uint8), off,
                                out_dtype=torch.float32)
        assert torch.equal(got.double(), base.double() * 2.0 ** (ka + kw)), (ka, kw)


def test_empty_and_types(gpu):
    from combine_moe_route_gb300 import binding as b
    q, s = b.quantize_mx4(torch.empty((0, 64), dtype=torch.bfloat16, device=gpu))
    assert q.shape == (0, 32) and s.shape == (0, 2) and b.dequantize_mx4(q, s).shape == (0, 64)
    w, sw = b.quantize_mx4(torch.ones((2, 64, 64), device=gpu))
    off = torch.zeros(3, dtype=torch.int32, device=gpu)
    assert b.expert_gemm_mx4(q, s, w, sw, off).shape == (0, 64)
    assert b.expert_gated_gemm_mx4(q, s, w, sw, off).q.shape == (0, 16)
    a, sa = b.quantize_mx4(torch.ones((3, 64), device=gpu))
    off = torch.tensor([0, 1, 3], dtype=torch.int32, device=gpu)
    want = b.expert_gemm_mx4(a, sa, w, sw, off)
    assert (want == 64).all()
    if hasattr(torch, "float4_e2m1fn_x2") and hasattr(torch, "float8_e8m0fnu"):
        f4, e8 = torch.float4_e2m1fn_x2, torch.float8_e8m0fnu
        assert torch.equal(b.expert_gemm_mx4(a.view(f4), sa.view(e8), w.view(f4), sw.view(e8), off), want)


def test_other_stream_and_graph(gpu):
    from combine_moe_route_gb300 import binding as b
    gen = torch.Generator(device=gpu).manual_seed(0)
    x = torch.randn((300, 512), generator=gen, device=gpu, dtype=torch.bfloat16)
    w13, s13 = b.quantize_mx4(torch.randn((3, 256, 512), generator=gen, device=gpu))
    w2, s2 = b.quantize_mx4(torch.randn((3, 512, 128), generator=gen, device=gpu))
    off = torch.tensor([0, 100, 100, 300], dtype=torch.int32, device=gpu)

    def run(stream=None):
        q, s = b.quantize_mx4(x, stream=stream)
        g = b.expert_gated_gemm_mx4(q, s, w13, s13, off, stream=stream)
        return b.expert_gemm_mx4(g.q, g.scale, w2, s2, off, stream=stream)

    want = run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        assert torch.equal(run(side), want)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    for seed in range(3):
        x.copy_(torch.randn((300, 512), generator=gen, device=gpu))
        graph.replay()
        got = out.clone()
        assert torch.equal(got, run())
    assert b.get_expert_error()[0] == 0


def test_chained_calls_read_what_was_written_just_before(gpu):
    """Each step reads what the kernel before it wrote, at sizes whose launches overlap."""
    from combine_moe_route_gb300 import binding as b
    gen = torch.Generator(device=gpu).manual_seed(1)
    E, H, I, rows = 8, 512, 256, 1000
    w13, s13 = b.quantize_mx4(torch.randn((E, 2 * I, H), generator=gen, device=gpu))
    w2, s2 = b.quantize_mx4(torch.randn((E, H, I), generator=gen, device=gpu) * 0.01)
    off = torch.linspace(0, rows, E + 1, device=gpu).int()
    xs = [torch.randn((rows, H), generator=gen, device=gpu).bfloat16() for _ in range(4)]

    def layer(x):
        q, s = b.quantize_mx4(x)
        g = b.expert_gated_gemm_mx4(q, s, w13, s13, off)
        return b.expert_gemm_mx4(g.q, g.scale, w2, s2, off)

    apart = []
    for x in xs:
        torch.cuda.synchronize()
        apart.append(layer(x))
    torch.cuda.synchronize()
    for _ in range(5):
        together = [layer(x) for x in xs]
        for g, w in zip(together, apart):
            assert torch.equal(g, w)
