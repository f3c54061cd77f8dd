"""A mixture-of-experts layer whose experts are real products: gated experts in e4m3 with fp32
scales per 128 channels and per 128 x 128 block, from the router's logits to the combined output,
and the gradients of the tokens and the logits.

Forward: route -> FP8 dispatch -> gated first product (quantised by its own epilogue) -> second
product -> combine.  Backward: combine gradient (quantised) -> transposed second product -> gate
gradient (quantised) -> transposed first product -> dispatch gradient, with the router's gradient
from the combine's.  The weights are quantised parameters and get no gradient; the quantisations
pass gradients through unchanged.  Autograd records neither pass: a tensor that requires a gradient
gets none through ``expert_layer``, only from ``expert_layer_backward``.

``python -m combine_moe_route_gb300.experts`` runs one layer both ways on the GPU.
"""
from __future__ import annotations

from dataclasses import dataclass, fields, is_dataclass

import torch

from . import binding as _b


def quantize_blocks(w: torch.Tensor) -> tuple[torch.Tensor, torch.Tensor]:
    """Weights [..., N, C] to e4m3 and fp32 scales [..., ceil(N/128), ceil(C/128)], one per
    128 x 128 block: scale = amax / 448 (amax at least 2^-119).  Done once, when weights are loaded."""
    N, C = w.shape[-2:]
    nb, cb = -(-N // 128), -(-C // 128)
    blocks = torch.nn.functional.pad(w.float(), (0, cb * 128 - C, 0, nb * 128 - N))
    blocks = blocks.unflatten(-1, (cb, 128)).unflatten(-3, (nb, 128))          # [..., nb, 128, cb, 128]
    amax = blocks.abs().amax(dim=(-3, -1)).clamp(min=2.0 ** -119)
    q = (blocks * (448.0 / amax)[..., :, None, :, None]).clamp(-448.0, 448.0)
    q = q.flatten(-2, -1).flatten(-3, -2)[..., :N, :C]
    return q.to(torch.float8_e4m3fn).contiguous(), (amax / 448.0).contiguous()


@dataclass
class ExpertWeights:
    """The experts of a layer: w13 [E, 2I, H] holds each gate's I rows, then its up projection's;
    w2 [E, H, I]."""
    w13: torch.Tensor
    w13_scale: torch.Tensor
    w2: torch.Tensor
    w2_scale: torch.Tensor

    @classmethod
    def quantized(cls, w13: torch.Tensor, w2: torch.Tensor) -> "ExpertWeights":
        return cls(*quantize_blocks(w13), *quantize_blocks(w2))

    @property
    def E(self) -> int:
        return self.w13.shape[0]


@dataclass
class ExpertForward:
    out: torch.Tensor                   # [T, H]
    topk_idx: torch.Tensor
    topk_w: torch.Tensor
    dispatch: _b.DispatchResult
    gated: _b.GatedResult
    y: torch.Tensor                     # [T*K, H] bf16: the expert outputs


def _record(stream, *values) -> None:
    """Every tensor in ``values`` (in results and weights too) keeps its memory, once dropped, until
    what ``stream`` has been given by then is done."""
    for v in values:
        if is_dataclass(v):
            _record(stream, *(getattr(v, f.name) for f in fields(v)))
        elif isinstance(v, tuple):
            _record(stream, *v)
        elif getattr(v, "is_cuda", False):   # anything else is the bindings' to refuse
            v.record_stream(stream)


def _on(stream, inputs: tuple, run):
    """``run()`` with ``stream`` current (None: as it is), so that what a pass allocates belongs to the
    stream that it runs on: its temporaries are dropped while the stream has yet to reach them.  The
    inputs come from the caller's stream and the results go there; each may be dropped while the
    other stream still uses it."""
    if stream is None:
        return run()
    caller = torch.cuda.current_stream(stream.device)
    _record(stream, *inputs)
    with torch.cuda.stream(stream):
        result = run()
    _record(caller, result)
    return result


def expert_layer(x: torch.Tensor, logits: torch.Tensor, B, K: int, weights: ExpertWeights, *, train: bool = False,
                 out_dtype: torch.dtype = torch.bfloat16, stream=None) -> ExpertForward:
    """One layer: x [T, H] bf16 and logits [T, E] fp32 to the combined [T, H].  ``train`` keeps the
    pre-activations for ``expert_layer_backward``.  Everything is enqueued on ``stream`` (default: the
    current one), nothing synchronises: a given stream has to be ordered behind the work that writes
    the inputs, and whoever reads the results behind the stream."""
    E = weights.E
    if len(logits.shape) != 2 or logits.shape[1] != E:
        raise ValueError(f"logits must be [T, E] with a column for each of the weights' {E} experts, got "
                         f"{tuple(logits.shape)}")

    def run():
        idx, w = _b.route_topk(logits, K)
        d = _b.dispatch(x, idx, B, E, fp8=True)
        g = _b.expert_gated_gemm(d.recv_x, d.recv_scale, weights.w13, weights.w13_scale, d.expert_offsets,
                                 save_h=train)
        y = _b.expert_gemm(g.q, g.scale, weights.w2, weights.w2_scale, d.expert_offsets)
        out = _b.combine(y, d.tok2row, w, out_dtype=out_dtype)
        return ExpertForward(out, idx, w, d, g, y)

    return _on(stream, (x, logits, weights), run)


def expert_layer_backward(dout: torch.Tensor, fwd: ExpertForward, weights: ExpertWeights, *, stream=None):
    """(dx [T, H] bf16, dlogits [T, E] fp32) for dout [T, H] bf16 and a ``train`` forward; ``stream`` as
    there."""
    if fwd.gated.h is None:
        raise ValueError("the forward pass kept no pre-activations: run it with train=True")
    d, K = fwd.dispatch, fwd.topk_idx.shape[1]

    def run():
        c = _b.combine_backward(dout, fwd.y, d.tok2row, fwd.topk_w, topk_idx=fwd.topk_idx, E=weights.E, fp8=True)
        dv = _b.expert_gemm(c.dy, c.dy_scale, weights.w2, weights.w2_scale, d.expert_offsets, transpose=True)
        dh, dh_scale = _b.expert_gated_backward(fwd.gated.h, dv)
        drows = _b.expert_gemm(dh, dh_scale, weights.w13, weights.w13_scale, d.expert_offsets, transpose=True)
        return _b.dispatch_backward(drows, d.tok2row, K), c.dlogits

    return _on(stream, (dout, fwd, weights), run)


def main() -> None:
    T, H, inner, E, K, R = 512, 1024, 512, 32, 4, 8
    gen = torch.Generator(device="cuda").manual_seed(0)
    w13 = torch.randn((E, 2 * inner, H), generator=gen, device="cuda") / H ** 0.5
    w2 = torch.randn((E, H, inner), generator=gen, device="cuda") / inner ** 0.5
    weights = ExpertWeights.quantized(w13, w2)
    x = torch.randn((T, H), generator=gen, device="cuda").bfloat16()
    logits = torch.randn((T, E), generator=gen, device="cuda")
    B = [T // R] * R
    fwd = expert_layer(x, logits, B, K, weights, train=True)
    dx, dlogits = expert_layer_backward(torch.ones_like(fwd.out), fwd, weights)
    status, _ = _b.get_device_error(fwd.dispatch.workspace)
    print(f"{T} tokens, {E} experts, top-{K}: out {tuple(fwd.out.shape)} rms {fwd.out.float().square().mean().sqrt():.3f}, "
          f"dx rms {dx.float().square().mean().sqrt():.3f}, dlogits rms {dlogits.square().mean().sqrt():.4f}; "
          f"device status {status}, {_b.get_expert_error()[0]}")


if __name__ == "__main__":
    main()
