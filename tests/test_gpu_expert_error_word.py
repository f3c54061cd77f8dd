"""The products' error word between streams and readers: a time-out is reported once, by whichever
stream's read comes first, and never lost.  (A test-only build withholds one stage.)"""
import threading

import numpy as np
import pytest
import torch

import _expert_ref as ref

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


@pytest.fixture
def product():
    inp = ref.product_inputs([40], 128, 512, np.random.default_rng(1))
    args = [inp[k].to("cuda:0") for k in ("a", "a_scale", "w", "w_scale", "off")]
    torch.cuda.synchronize()
    return args


def test_one_word_for_all_streams(hooked, product):
    """A read on another stream, behind the failed product's, takes its error; the next finds none."""
    from combine_moe_route_gb300 import binding as b
    failing, other = torch.cuda.Stream(), torch.cuda.Stream()
    with b.using_library(hooked):
        assert b.get_expert_error() == (OK, 0)
        b.expert_gemm(*product, stream=failing)
        failing.synchronize()
        assert b.get_expert_error(stream=other) == (TIMEOUT, COPY_TIMEOUT)
        assert b.get_expert_error(stream=failing) == (OK, 0)


def test_readers_at_the_same_time(hooked, product):
    """Threads read on streams of their own while products fail: every failure is seen, and one
    failure by one reader only."""
    from combine_moe_route_gb300 import binding as b
    seen, stop = [[] for _ in range(4)], threading.Event()

    def read(log):
        stream = torch.cuda.Stream()
        while not stop.is_set():
            log.append(b.get_expert_error("cuda:0", stream=stream))

    with b.using_library(hooked):
        readers = [threading.Thread(target=read, args=(log,)) for log in seen]
        for t in readers:
            t.start()
        # its roles' waits run out at different times, each setting the bit: one or a few reports
        b.expert_gemm(*product)
        torch.cuda.synchronize()
        stop.set()
        for t in readers:
            t.join()
        last = b.get_expert_error()
        reports = sum(log.count((TIMEOUT, COPY_TIMEOUT)) for log in seen) + (last != (OK, 0))
        blocks, roles = 8, 12   # at most: a cluster's blocks and their warps
        assert 1 <= reports <= blocks * roles
        assert all(r in ((OK, 0), (TIMEOUT, COPY_TIMEOUT)) for log in seen for r in log)
        assert b.get_expert_error() == (OK, 0)
