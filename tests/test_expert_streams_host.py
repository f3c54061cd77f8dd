"""The layer on a stream that is not the current one, without a GPU: every call of a pass, and so
every allocation in it, is made with that stream current, and what the caller's stream and the
layer's stream use of each other's memory is recorded."""
from contextlib import contextmanager
from types import SimpleNamespace

import pytest
import torch

from combine_moe_route_gb300 import experts


class Handed:
    """Stands for a tensor: remembers the streams its memory is recorded on."""
    is_cuda = True

    def __init__(self, *shape):
        self.shape, self.streams = shape, []

    def dim(self):
        return len(self.shape)

    def record_stream(self, s):
        self.streams.append(s)


@pytest.fixture
def traced(monkeypatch):
    """The bindings replaced by recorders of the current stream."""
    current, calls, made = ["caller"], [], []

    @contextmanager
    def stream_context(s):
        if s is not None:
            current.append(s)
        yield
        if s is not None:
            current.pop()

    def new(*shape):
        t = Handed(*shape)
        made.append(t)
        return t

    def call(name, result):
        def f(*args, stream=None, **kwargs):
            calls.append((name, current[-1] if stream is None else stream, current[-1]))
            return result()
        return f

    b = experts._b
    for name, result in (
            ("route_topk", lambda: (new(4, 2), new(4, 2))),
            ("dispatch", lambda: b.DispatchResult(*(new(8, 128) for _ in range(8)))),
            ("expert_gated_gemm", lambda: b.GatedResult(new(8, 128), new(8, 1), new(8, 256))),
            ("expert_gemm", lambda: new(8, 128)), ("combine", lambda: new(4, 128)),
            ("combine_backward", lambda: b.CombineGrad(*(new(8, 128) for _ in range(4)))),
            ("expert_gated_backward", lambda: (new(8, 256), new(8, 2))), ("dispatch_backward", lambda: new(4, 128))):
        monkeypatch.setattr(b, name, call(name, result))
    monkeypatch.setattr(torch.cuda, "stream", stream_context)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: current[-1])
    return SimpleNamespace(calls=calls, made=made, current=current)


def _layer(stream):
    w = experts.ExpertWeights(Handed(3, 256, 128), Handed(3, 2, 1), Handed(3, 128, 128), Handed(3, 1, 1))
    x, logits, dout = Handed(4, 128), Handed(4, 3), Handed(4, 128)
    f = experts.expert_layer(x, logits, [4], 2, w, train=True, stream=stream)
    grads = experts.expert_layer_backward(dout, f, w, stream=stream)
    return (x, logits, dout, w.w13, w.w13_scale, w.w2, w.w2_scale), f, grads


def test_allocations_and_kernels_are_on_one_stream(traced):
    side = SimpleNamespace(device="cuda:0")
    inputs, f, grads = _layer(side)
    assert len(traced.calls) == 10 and traced.current == ["caller"]
    for name, ran_on, allocated_on in traced.calls:
        assert ran_on is side and allocated_on is side, name
    for t in inputs:                     # the caller may drop them while the stream still reads them
        assert side in t.streams
    results = [f.out, f.topk_idx, f.topk_w, f.y, f.gated.q, f.gated.h, f.dispatch.recv_x, f.dispatch.workspace, *grads]
    for t in results:                    # ... and the caller's stream may still read the results when they go
        assert "caller" in t.streams
    for t in (f.y, f.topk_w, f.gated.h, f.dispatch.tok2row):   # read again by the backward pass
        assert side in t.streams


def test_the_current_stream_records_nothing(traced):
    _layer(None)
    assert len(traced.calls) == 10 and all(c[1] == c[2] == "caller" for c in traced.calls)
    assert not any(t.streams for t in traced.made)
