"""Sizes past what a launch can cover are refused, without a GPU (nothing is enqueued)."""
import pytest

INVALID = 1
BF16, FP8 = 0, 1
FAKE = 0x100000      # never dereferenced: every call below is refused


@pytest.fixture(scope="module")
def lib():
    from combine_moe_route_gb300 import binding, build
    build.build()
    return binding.load_library()


@pytest.mark.parametrize("dtype", [BF16, FP8])
@pytest.mark.parametrize("rows,I", [(2 ** 31 - 1, 32768), (2 ** 31 - 1, 2048 + 128), (2 ** 27 + 1, 32768)])
def test_gated_backward_past_the_grid(lib, rows, I, dtype):
    assert lib.moe_expert_gated_backward(FAKE, FAKE, rows, I, dtype, FAKE, FAKE, None) == INVALID
