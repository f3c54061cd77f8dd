"""Failure detection of the 4-bit products without a GPU fault: in a test-only build the loading warp
withholds one stage, so every role's bounded wait runs out.  The kernel returns, the error word says
so and is cleared by the read, nothing outside the output is written, and the context stays usable."""
import numpy as np
import pytest
import torch

import _mx4_ref as ref

pytestmark = pytest.mark.gpu

OK, TIMEOUT, COPY_TIMEOUT = 0, 5, 0x8


@pytest.fixture(scope="module")
def hooked(tmp_path_factory):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from combine_moe_route_gb300 import binding, build
    build.build()
    out = str(tmp_path_factory.mktemp("withheld"))
    return binding.load_library(build.build(out_dir=out, defines=("MOE_TEST_WITHHOLD_PRODUCT_STAGE=1",)))


# blocks that share a tile's channels; single blocks (of many tiles); pairs and a tail of 44 rows
@pytest.mark.parametrize("counts,C", [([20], 2048), ([1] * 100, 512), ([1600], 512)])
def test_a_stage_that_never_comes(hooked, counts, C):
    from combine_moe_route_gb300 import binding as b
    gpu = torch.device("cuda:0")
    inp = ref.product_inputs(counts, 256, C, np.random.default_rng(0))
    args = [inp[k].to(gpu) for k in ("a", "a_scale", "w", "w_scale", "off")]
    rows = sum(counts)
    big = torch.full((rows + 200, 256), 7.0, device=gpu)
    out = big[100:100 + rows]
    want = b.expert_gemm_mx4(*args, out_dtype=torch.float32)
    assert b.get_expert_error() == (OK, 0)
    with b.using_library(hooked):
        b.expert_gemm_mx4(*args, out=out)
        assert b.get_expert_error() == (TIMEOUT, COPY_TIMEOUT)
        assert b.get_expert_error() == (OK, 0)
    assert (big[:100] == 7).all() and (big[100 + rows:] == 7).all()
    b.expert_gemm_mx4(*args, out=out)
    assert b.get_expert_error() == (OK, 0) and torch.equal(out, want)
