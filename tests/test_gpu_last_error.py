"""A call that fails leaves no error behind for the calls after it."""
import ctypes

import pytest
import torch

pytestmark = pytest.mark.gpu

OK, CUDA_ERROR = 0, 3


@pytest.fixture(scope="module")
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from combine_moe_route_gb300 import build
    build.build()
    return torch.device("cuda:0")


@pytest.mark.parametrize("reader", ["moe_get_expert_error", "moe_get_device_error"])
def test_a_failed_read_does_not_fail_the_next_call(gpu, reader):
    """The synchronous readers cannot run while their stream is captured: the read says so, the
    capture is void, and a combine on another stream afterwards is none the worse."""
    from combine_moe_route_gb300 import binding as b
    lib = b.load_library()
    y, w = torch.ones((4, 8), dtype=torch.bfloat16, device=gpu), torch.ones((4, 1), device=gpu)
    out = torch.zeros((4, 8), dtype=torch.bfloat16, device=gpu)
    ws = torch.zeros(4096, dtype=torch.uint8, device=gpu)
    captured, other = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    code = ctypes.c_int32(0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(captured):
        graph.capture_begin(capture_error_mode="relaxed")
        if reader == "moe_get_expert_error":
            read = lib.moe_get_expert_error(ctypes.byref(code), captured.cuda_stream)
        else:
            read = lib.moe_get_device_error(ws.data_ptr(), ctypes.byref(code), captured.cuda_stream)
        combined = lib.moe_combine(y.data_ptr(), None, w.data_ptr(), 4, 1, 8, 0, out.data_ptr(), other.cuda_stream)
        with pytest.raises(RuntimeError):
            graph.capture_end()
    torch.cuda.synchronize()
    assert read == CUDA_ERROR and code.value == 0
    assert combined == OK
    assert (out == 1).all()
    assert b.get_expert_error() == (0, 0)
