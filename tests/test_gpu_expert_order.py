"""Products directly behind the kernel that writes what they read: both launches of a call with
many rows (the pairs and the tails) see the rows, scales and offsets of the kernel before."""
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


@pytest.mark.parametrize("gated", [False, True])
def test_products_see_what_the_kernel_before_wrote(gpu, gated):
    """A gradient kernel overwrites the product's rows and scales, a copy its offsets, call after
    call without a wait of the host; every result equals the one of the same calls with waits."""
    from combine_moe_route_gb300 import binding as b
    T, K, H, N, E, calls = 1500, 2, 512, 512, 4, 30
    rows = T * K
    gen = torch.Generator(device=gpu).manual_seed(0)
    w = torch.randn((E, N, H), generator=gen, device=gpu).mul_(60).clamp_(-448, 448).to(torch.float8_e4m3fn)
    w_scale = torch.rand((E, N // 128, H // 128), generator=gen, device=gpu) * 1e-3
    dout = torch.randn((calls, T, H), generator=gen, device=gpu).bfloat16()
    y = torch.randn((rows, H), generator=gen, device=gpu).bfloat16()
    at = torch.randperm(rows, generator=gen, device=gpu).int()
    topk_w = torch.rand((T, K), generator=gen, device=gpu) + 0.1
    # every expert ends in a rest of 1 to 128 rows, another one in every call
    cut = torch.tensor([[0, 256 + i, 768 + 3 * i, 1792 + 4 * i, rows] for i in range(1, calls + 1)], dtype=torch.int32)
    cut = cut.to(gpu)
    dy = torch.empty((rows, H), dtype=torch.float8_e4m3fn, device=gpu)
    dy_scale = torch.empty((rows, H // 128), device=gpu)
    off = torch.empty(E + 1, dtype=torch.int32, device=gpu)

    def run(wait):
        results = []
        for i in range(calls):
            off.copy_(cut[i])
            b.combine_backward(dout[i], y, at, topk_w, fp8=True, out=dy, out_scale=dy_scale)
            if wait:
                torch.cuda.synchronize()
            if gated:
                r = b.expert_gated_gemm(dy, dy_scale, w, w_scale, off)
                results += [r.q.view(torch.uint8), r.scale]
            else:
                results.append(b.expert_gemm(dy, dy_scale, w, w_scale, off))
            if wait:
                torch.cuda.synchronize()
        return results

    want, got = run(True), run(False)
    assert b.get_expert_error() == (0, 0)
    for i, (a, c) in enumerate(zip(want, got)):
        assert torch.equal(a, c), i
