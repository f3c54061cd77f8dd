"""Products at the ends of their ranges: scales whose product leaves the normal numbers, an fp32
result of more than 2^31 bytes from pairs and tails, and two streams of products at once."""
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


def _to(gpu, inp):
    return [inp[k].to(gpu) for k in ("a", "a_scale", "w", "w_scale", "off")]


@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("C", [128, 640, 2048])
def test_tiny_scales(gpu, C, transpose):
    """Scales from the quantiser's smallest, 2^-128, up: a row's times a weight's is formed first, and
    below 2^-126 is a multiple of 2^-149, so half of that times the block's sum of products may be
    off; the sums themselves are multiples of 2^-149 there."""
    from combine_moe_route_gb300 import binding as b
    counts, N = [5, 0, 40, 130], 144
    rng = np.random.default_rng(C)
    inp = ref.product_inputs(counts, N, C, rng, transpose)
    inp["a_scale"] = torch.from_numpy(np.exp2(rng.uniform(-128, -96, inp["a_scale"].shape)).astype(np.float32))
    inp["w_scale"] = torch.from_numpy(np.exp2(rng.uniform(-24, -8, inp["w_scale"].shape)).astype(np.float32))
    want, mag = ref.product(inp, transpose)
    ones = dict(inp, a_scale=torch.ones_like(inp["a_scale"]), w_scale=torch.ones_like(inp["w_scale"]))
    _, codes = ref.product(ones, transpose)
    bound = ref.product_bound(mag, C) + 2.0 ** -150 * (codes + ref.blocks(C) + 2)
    o32 = b.expert_gemm(*_to(gpu, inp), transpose=transpose, out_dtype=torch.float32).cpu().double()
    o16 = b.expert_gemm(*_to(gpu, inp), transpose=transpose).cpu().double()
    assert ((o32 - want).abs() <= bound).all()
    assert ((o16 - want).abs() <= bound + 2.0 ** -8 * want.abs() + 2.0 ** -134).all()
    assert float((o32 - want).norm() / want.norm()) < 1e-6


def test_fp32_result_past_32_bits_from_pairs_and_tails(gpu):
    """A result of 2.4e9 values, 9.6e9 bytes: the first rows, those around its 2^31st byte and value,
    and the last, a rest of 71 rows."""
    from combine_moe_route_gb300 import binding as b
    N, C = 7168, 144
    gen = torch.Generator(device=gpu).manual_seed(11)
    counts = [131_072, 70, 204_800 + 71]
    rows = sum(counts)
    a = torch.randn((rows, C), generator=gen, device=gpu).to(torch.float8_e4m3fn)
    sa = torch.rand((rows, 2), generator=gen, device=gpu) + 0.5
    w = torch.randn((3, N, C), generator=gen, device=gpu).to(torch.float8_e4m3fn)
    sw = torch.rand((3, N // 128, 2), generator=gen, device=gpu) + 0.5
    off = torch.tensor([0, counts[0], counts[0] + counts[1], rows], dtype=torch.int32, device=gpu)
    out = b.expert_gemm(a, sa, w, sw, off, out_dtype=torch.float32)
    byte, value = 2 ** 31 // (4 * N), 2 ** 31 // N
    for lo, hi, e in ((0, 130, 0), (byte - 1, byte + 2, 0), (counts[0], counts[0] + 70, 1), (value - 1, value + 2, 2),
                      (rows - 200, rows, 2)):
        assert off[e] <= lo and hi <= off[e + 1]
        inp = dict(a=a[lo:hi].cpu(), a_scale=sa[lo:hi].cpu(), w=w[e:e + 1].cpu(), w_scale=sw[e:e + 1].cpu(),
                   off=torch.tensor([0, hi - lo]))
        want, mag = ref.product(inp)
        assert ((out[lo:hi].cpu().double() - want).abs() <= ref.product_bound(mag, C)).all()


def test_two_streams_of_products(gpu):
    """Products of every form at once on two streams: each as alone, bit for bit."""
    from combine_moe_route_gb300 import binding as b
    sets = []
    for i, counts in enumerate(([300, 520, 90, 700], [3, 0, 1, 8])):        # pairs and tails; shared channels
        inp = ref.product_inputs(counts, 512, 2048, np.random.default_rng(i))
        args = _to(gpu, inp)
        sets.append((args, b.expert_gemm(*args), b.expert_gated_gemm(*args)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    outs = [[(torch.empty_like(y), b.GatedResult(torch.empty_like(g.q), torch.empty_like(g.scale), None))
             for _ in range(20)] for _, y, g in sets]
    torch.cuda.synchronize()
    for i in range(20):
        for (args, _, _), st, o in zip(sets, streams, outs):
            b.expert_gemm(*args, out=o[i][0], stream=st)
            b.expert_gated_gemm(*args, out=o[i][1].q, out_scale=o[i][1].scale, stream=st)
    torch.cuda.synchronize()
    assert b.get_expert_error() == (0, 0)
    for (_, y, g), o in zip(sets, outs):
        for oy, og in o:
            assert torch.equal(oy, y) and torch.equal(og.scale, g.scale)
            assert torch.equal(og.q.view(torch.uint8), g.q.view(torch.uint8))
