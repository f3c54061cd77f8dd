"""The combine's forms at more tokens than a grid has blocks for: the blocks walk the rest."""
import pytest
import torch

pytestmark = pytest.mark.gpu

T, H = 2 ** 30, 8


@pytest.fixture(scope="module")
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    if torch.cuda.mem_get_info()[0] < 60e9:
        pytest.skip("needs 50 GB")
    from combine_moe_route_gb300 import build
    build.build()
    return torch.device("cuda:0")


@pytest.mark.parametrize("form", ["combine", "combine_recv", "dispatch_backward"])
def test_a_billion_tokens(gpu, form):
    """2^30 tokens of 8 channels, one expert each: token g takes row g + 5, with weight 1."""
    from combine_moe_route_gb300 import binding as b
    y = torch.empty((T, H), dtype=torch.bfloat16, device=gpu)
    bits = torch.arange(64 * H, dtype=torch.int16, device=gpu) + 0x3f80    # 512 values of 1 and more
    y.view(torch.int16).view(-1, 64 * H).copy_(bits)
    at = torch.arange(5, T + 5, dtype=torch.int32, device=gpu)
    at[-5:] -= T
    out = torch.full((T, H), -1.0, dtype=torch.bfloat16, device=gpu)
    if form == "dispatch_backward":
        b.dispatch_backward(y, at, 1, out=out)
    else:
        w = torch.ones((T, 1), device=gpu)
        if form == "combine":
            b.combine(y, at, w, out=out)
        else:
            ws = torch.zeros(1 << 16, dtype=torch.uint8, device=gpu)
            b.combine_send(ws, 1)
            b.combine_recv(y, at, w, ws, 1, out=out)
            assert b.get_device_error(ws) == (0, 0)
    same = torch.equal(out[:-5], y[5:]) and torch.equal(out[-5:], y[:5])
    del y, at, out
    torch.cuda.empty_cache()
    assert same
