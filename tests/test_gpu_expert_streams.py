"""The layer on another stream than the caller's: its temporaries are its own for as long as the
stream runs, whatever the caller allocates, writes or drops meanwhile."""
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


def test_layer_on_a_side_stream(gpu):
    """The side stream is busy when a pass is enqueued; the caller fills new tensors of every
    size the pass has, drops the forward's results, and reads the gradients after a join."""
    import combine_moe_route_gb300 as moe
    T, H, inner, E, K, B = 2048, 512, 256, 8, 2, [1500, 548]
    gen = torch.Generator(device=gpu).manual_seed(3)
    w = moe.ExpertWeights.quantized(torch.randn((E, 2 * inner, H), generator=gen, device=gpu) / H ** 0.5,
                                    torch.randn((E, H, inner), generator=gen, device=gpu) / inner ** 0.5)
    x = torch.randn((T, H), generator=gen, device=gpu).bfloat16()
    logits = torch.randn((T, E), generator=gen, device=gpu)
    dout = torch.randn((T, H), generator=gen, device=gpu).bfloat16()
    f = moe.expert_layer(x, logits, B, K, w, train=True)
    want_out = f.out.clone()
    want_dx, want_dl = moe.expert_layer_backward(dout, f, w)
    del f
    busy = torch.randn((4096, 4096), generator=gen, device=gpu).bfloat16()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(5):
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            for _ in range(20):
                torch.mm(busy, busy)
        f = moe.expert_layer(x, logits, B, K, w, train=True, stream=side)
        out = f.out
        dx, dl = moe.expert_layer_backward(dout, f, w, stream=side)
        del f
        rows = T * K
        fill = [torch.full(shape, 77, dtype=t, device=gpu)
                for shape, t in (((rows, H), torch.uint8), ((rows, H), torch.bfloat16), ((rows, inner), torch.bfloat16),
                                 ((rows, 2 * inner), torch.bfloat16), ((rows, 2 * inner), torch.uint8),
                                 ((rows, H // 128), torch.float32), ((T, K), torch.float32), ((T, E), torch.float32))
                for _ in range(3)]
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(out, want_out) and torch.equal(dx, want_dx) and torch.equal(dl, want_dl)
        assert all((v == 77).all() for v in fill)
    assert moe.get_expert_error() == (0, 0)


def test_layer_on_a_forked_stream_in_a_graph(gpu):
    """Captured on a stream forked from the capturing one, and replayed."""
    import combine_moe_route_gb300 as moe
    T, H, inner, E, K = 64, 256, 128, 4, 2
    gen = torch.Generator(device=gpu).manual_seed(4)
    w = moe.ExpertWeights.quantized(torch.randn((E, 2 * inner, H), generator=gen, device=gpu) / H ** 0.5,
                                    torch.randn((E, H, inner), generator=gen, device=gpu) / inner ** 0.5)
    x = torch.randn((T, H), generator=gen, device=gpu).bfloat16()
    logits = torch.randn((T, E), generator=gen, device=gpu)
    dout = torch.randn((T, H), generator=gen, device=gpu).bfloat16()
    f = moe.expert_layer(x, logits, [T], K, w, train=True)
    dx, dl = moe.expert_layer_backward(dout, f, w)
    torch.cuda.synchronize()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        f2 = moe.expert_layer(x, logits, [T], K, w, train=True, stream=side)
        dx2, dl2 = moe.expert_layer_backward(dout, f2, w, stream=side)
        torch.cuda.current_stream().wait_stream(side)
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(f2.out, f.out) and torch.equal(dx2, dx) and torch.equal(dl2, dl)
