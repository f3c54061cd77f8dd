"""Cases, plain forms and calls of the expert-side operators, for timing and comparison.

Five operators around the dispatch and the combine of a mixture-of-experts layer:

* ``expert_gemm``: the experts' product over the rows dispatch leaves grouped by expert, in
  e4m3 with one fp32 scale per 128 channels of a row and per 128 x 128 block of a weight;
  forward (out = a w^T) and for the gradient of its input (out = a w, ``transpose``).
* ``expert_gated_gemm``: the first product of a gated expert with silu(gate) * up and the
  quantisation of its result in one pass.
* ``expert_gated_backward``: the gradient of that gate, quantised for the transposed product.
* ``combine_backward``: the gradient of the weighted sum over a token's experts, to the expert
  outputs, the routing weights and the router's logits.
* ``dispatch_backward``: the gradient of the scatter, a token's sum over its K copies.

With ``own`` false ``run`` computes an operator from elementary torch operations in 32 bits;
with ``own`` true it calls this package.
"""
import math

import torch

own = False

E4M3_MAX = 448.0
AMAX_FLOOR = 2.0 ** -119   # the smallest power of two whose 448 / amax is finite in fp32


def listed():
    return [
        # one token of a decode step: its 8 experts' second product, bound by reading 8 weights
        dict(name="gemm_token", op="gemm", T=1, E=256, top=8, N=7168, C=2048, zipf=0.0, transpose=False),
        # a decode step with skewed expert load (some experts idle, one with many rows)
        dict(name="gemm_skewed_decode", op="gemm", T=1003, E=384, top=8, N=7168, C=2048, zipf=1.2, transpose=False),
        # the second product of a prefill layer: 4096 tokens on each of 8 ranks
        dict(name="gemm_prefill", op="gemm", T=32768, E=256, top=8, N=7168, C=2048, zipf=0.0, transpose=False),
        # the gradient of the first product's input over a quarter of that batch
        dict(name="gemm_prefill_dx", op="gemm", T=8192, E=256, top=8, N=7168, C=4096, zipf=0.0, transpose=True),
        # one token's gated first product
        dict(name="gated_token", op="gated", T=1, E=256, top=8, I=2048, C=7168, zipf=0.0, save=False),
        # the gated first product of the prefill layer; pre-activations kept for a backward pass
        dict(name="gated_prefill", op="gated", T=32768, E=256, top=8, I=2048, C=7168, zipf=0.0, save=True),
        # the gate's gradient at a decode-sized batch, bf16
        dict(name="gated_backward_small", op="gated_backward", rows=8024, I=2048, fp8=False),
        # the gate's gradient over the prefill layer's rows, quantised for the next product
        dict(name="gated_backward_prefill", op="gated_backward", rows=262144, I=2048, fp8=True),
        # the toy layer, where the call's own cost counts: 2 of 16 experts, 259 tokens
        dict(name="combine_backward_toy", op="combine_backward", T=259, E=16, top=2, H=256, fp8=False),
        # the prefill layer's weighted sum, back to quantised rows and to the router's logits
        dict(name="combine_backward_prefill", op="combine_backward", T=32768, E=256, top=8, H=7168, fp8=True),
        # a decode-sized scatter's gradient, an odd number of tokens
        dict(name="dispatch_backward_decode", op="dispatch_backward", T=1003, E=256, top=8, H=7168),
        # the prefill layer's scatter
        dict(name="dispatch_backward_prefill", op="dispatch_backward", T=32768, E=256, top=8, H=7168),
    ]


_WIDE = (256, 512, 640, 1152, 1664, 2048, 2432, 4096, 5120, 7168)     # multiples of 128
_RAGGED = (208, 400, 720, 1328, 2000, 2880, 4240)                     # multiples of 16 only


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gemm", "gemm", "gated", "gated_backward", "combine_backward", "dispatch_backward"])
    if op in ("gemm", "gated"):
        E = rng.choice([8, 16, 32, 64, 128, 256])
        top = rng.choice([1, 2, 3, 4, 6, 8])
        zipf = rng.choice([0.0, 0.0, 0.0, 0.7, 1.2])
        T = _log_int(rng, 1, 2048 if zipf else 32768) | 1
        if op == "gemm":
            N, C = rng.choice(_WIDE + _RAGGED), rng.choice(_WIDE + _RAGGED)
            case = dict(op="gemm", T=T, E=E, top=top, N=N, C=C, zipf=zipf, transpose=rng.random() < 0.5)
        else:
            case = dict(op="gated", T=T, E=E, top=top, I=rng.choice(_WIDE[:6]), C=rng.choice(_WIDE), zipf=zipf,
                        save=rng.random() < 0.5)
            N, C = 2 * case["I"], case["C"]
        while 2.0 * case["T"] * top * N * C > 4e12 or E * (4.0 * case["T"] * top / E + 64) * C * 4 > 2e10:
            case["T"] = (case["T"] // 2) | 1
        return case
    if op == "gated_backward":
        return dict(op=op, rows=_log_int(rng, 1, 131072) | 1, I=rng.choice(_WIDE[:6]), fp8=rng.random() < 0.5)
    E = rng.choice([8, 16, 60, 64, 128, 256, 384])
    case = dict(op=op, T=_log_int(rng, 1, 32768) | 1, E=E, top=rng.choice([1, 2, 3, 4, 6, 8]), H=rng.choice(_WIDE))
    if op == "combine_backward":
        case["fp8"] = rng.random() < 0.5
    return case


# --------------------------------------------------------------------------- inputs

def _route(case, gen, dev):
    """Logits, the top experts by descending logit, their softmax weights, and the grouped rows."""
    T, E, top = case["T"], case["E"], case["top"]
    logits = torch.randn((T, E), generator=gen, device=dev)
    if case.get("zipf", 0.0):   # the log of a Zipf weight over a random order of the experts
        order = torch.randperm(E, generator=gen, device=dev).float()
        logits = logits - case["zipf"] * torch.log1p(order)
    w, idx = torch.sort(logits, dim=1, descending=True, stable=True)
    w, idx = torch.softmax(w[:, :top], dim=1).contiguous(), idx[:, :top].contiguous()
    row2src = torch.sort(idx.reshape(-1), stable=True).indices
    tok2row = torch.empty_like(row2src)
    tok2row[row2src] = torch.arange(T * top, device=dev)
    offsets = torch.zeros(E + 1, dtype=torch.int64, device=dev)
    offsets[1:] = torch.cumsum(torch.bincount(idx.reshape(-1), minlength=E), 0)
    return idx.int(), w, offsets, tok2row, row2src


def _blocks(n):
    return -(-n // 128)


def _quantize(v):
    """fp32 [n, C] -> e4m3 [n, C] and fp32 scales [n, ceil(C / 128)], the rule of the dispatch."""
    n, C = v.shape
    pad = torch.nn.functional.pad(v, (0, _blocks(C) * 128 - C)).view(n, _blocks(C), 128)
    amax = pad.abs().amax(2).clamp(min=AMAX_FLOOR)
    q = (pad * (E4M3_MAX / amax)[:, :, None]).clamp(-E4M3_MAX, E4M3_MAX)
    return q.view(n, -1)[:, :C].to(torch.float8_e4m3fn).contiguous(), amax / E4M3_MAX


def _take_rows(q, at):
    """q[at] of e4m3 values."""
    return q.view(torch.uint8)[at].view(torch.float8_e4m3fn)


def _weights(E, N, C, gen, dev):
    """Normal weights as their quantisation leaves them: about 4.2 sigma of a block at 448."""
    q = torch.empty((E, N, C), dtype=torch.float8_e4m3fn, device=dev)
    for e in range(0, E, 32):
        v = torch.randn(q[e:e + 32].shape, generator=gen, device=dev, dtype=torch.bfloat16)
        q[e:e + 32] = v.mul_(106.0).clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    u = torch.rand((E, _blocks(N), _blocks(C)), generator=gen, device=dev)
    return q, (0.8 + 0.4 * u) * (1.9 / 106.0 / math.sqrt(C))


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    s = dict(case=case)
    op = case["op"]
    if op in ("gemm", "gated"):
        T, E, top, C = case["T"], case["E"], case["top"], case["C"]
        N = case["N"] if op == "gemm" else 2 * case["I"]
        _, _, offsets, _, row2src = _route(case, gen, dev)
        # the copies of a token are the same row where it is dispatched (the gated first product);
        # the second product and the gradients have rows of their own
        if op == "gated":
            x = torch.randn((T, C), generator=gen, device=dev).bfloat16().float()
            q, scale = _quantize(x)
            s["a"], s["a_scale"] = _take_rows(q, row2src // top), scale[row2src // top].contiguous()
        else:
            s["a"] = torch.empty((T * top, C), dtype=torch.float8_e4m3fn, device=dev)
            s["a_scale"] = torch.empty((T * top, _blocks(C)), device=dev)
            for r in range(0, T * top, 65536):
                n = min(65536, T * top - r)
                v = torch.randn((n, C), generator=gen, device=dev)
                v = torch.nn.functional.silu(v) * torch.randn((n, C), generator=gen, device=dev)
                s["a"][r:r + n], s["a_scale"][r:r + n] = _quantize(v)
        wshape = (E, C, N) if case.get("transpose") else (E, N, C)
        s["w"], s["w_scale"] = _weights(*wshape, gen, dev)
        # the rows' bounds, and the experts that have any with the fullest one's count
        counts = torch.diff(offsets)
        s["offsets"], s["hit"], s["most"] = offsets.int(), torch.nonzero(counts).view(-1), int(counts.max())
        rows = T * top
        if op == "gemm":
            s["out"] = torch.empty((rows, N), dtype=torch.bfloat16, device=dev)
        else:
            s["q"] = torch.empty((rows, case["I"]), dtype=torch.float8_e4m3fn, device=dev)
            s["q_scale"] = torch.empty((rows, case["I"] // 128), device=dev)
            s["h"] = torch.empty((rows, N), dtype=torch.bfloat16, device=dev) if case["save"] else None
    elif op == "gated_backward":
        rows, inner = case["rows"], case["I"]
        s["h"] = torch.randn((rows, 2 * inner), generator=gen, device=dev).mul_(1.9).bfloat16()
        s["da"] = torch.randn((rows, inner), generator=gen, device=dev).mul_(1e-3).bfloat16()
        s["dh"] = torch.empty((rows, 2 * inner), dtype=torch.float8_e4m3fn if case["fp8"] else torch.bfloat16, device=dev)
        s["dh_scale"] = torch.empty((rows, 2 * inner // 128), device=dev) if case["fp8"] else None
    else:
        T, E, top, H = case["T"], case["E"], case["top"], case["H"]
        idx, w, _, tok2row, _ = _route(case, gen, dev)
        s["idx"], s["w"], s["tok2row"] = idx, w, tok2row.int()
        s["rows"] = torch.randn((T * top, H), generator=gen, device=dev, dtype=torch.bfloat16)
        if op == "combine_backward":
            s["dout"] = torch.randn((T, H), generator=gen, device=dev).mul_(1e-3).bfloat16()
            s["dy"] = torch.empty((T * top, H), dtype=torch.float8_e4m3fn if case["fp8"] else torch.bfloat16, device=dev)
            s["dy_scale"] = torch.empty((T * top, H // 128), device=dev) if case["fp8"] else None
            s["dw"], s["dlogits"] = torch.empty((T, top), device=dev), torch.empty((T, E), device=dev)
        else:
            s["dx"] = torch.empty((T, H), dtype=torch.bfloat16, device=dev)
    return s


# --------------------------------------------------------------------------- one pass

def run(state):
    return _own(state) if own else _plain(state)


def _own(s):
    import combine_moe_route_gb300 as moe
    case = s["case"]
    if case["op"] == "gemm":
        return moe.expert_gemm(s["a"], s["a_scale"], s["w"], s["w_scale"], s["offsets"],
                               transpose=case["transpose"], out=s["out"])
    if case["op"] == "gated":
        r = moe.expert_gated_gemm(s["a"], s["a_scale"], s["w"], s["w_scale"], s["offsets"],
                                  out=s["q"], out_scale=s["q_scale"], h=s["h"])
        return [r.q, r.scale] + ([r.h] if case["save"] else [])
    if case["op"] == "gated_backward":
        dh, scale = moe.expert_gated_backward(s["h"], s["da"], fp8=case["fp8"], out=s["dh"], out_scale=s["dh_scale"])
        return [dh, scale] if case["fp8"] else [dh]
    if case["op"] == "combine_backward":
        r = moe.combine_backward(s["dout"], s["rows"], s["tok2row"], s["w"], topk_idx=s["idx"], E=case["E"],
                                 fp8=case["fp8"], out=s["dy"], out_scale=s["dy_scale"], dtopk_w=s["dw"],
                                 dlogits=s["dlogits"])
        return [r.dy, r.dtopk_w, r.dlogits] + ([r.dy_scale] if case["fp8"] else [])
    return moe.dispatch_backward(s["rows"], s["tok2row"], case["top"], out=s["dx"])


def _spread(scale, *shape):
    """Scales per 128 of the last dimensions, repeated over their blocks."""
    for d in range(1, len(shape)):
        if scale.shape[d] != shape[d]:
            scale = scale.repeat_interleave(128, d).narrow(d, 0, shape[d])
    return scale


def _grouped_product(s):
    """fp32 rows of each expert times its weight: experts padded to the fullest, one batched product."""
    rows, C = s["a"].shape
    hit, most, dev = s["hit"], s["most"], s["a"].device
    first, end = s["offsets"].long()[hit], s["offsets"].long()[hit + 1]
    a = s["a"].float().mul_(_spread(s["a_scale"], rows, C))
    w = _take_rows(s["w"], hit).float()
    w.mul_(_spread(s["w_scale"][hit], *w.shape))
    padded = a[(first[:, None] + torch.arange(most, device=dev)).clamp(max=rows - 1)]
    out = torch.bmm(padded, w if s["case"].get("transpose") else w.transpose(1, 2))
    row = torch.arange(rows, device=dev)
    e = torch.searchsorted(end, row, right=True)
    return out.view(hit.numel() * most, -1)[e * most + row - first[e]]


def _plain(s):
    case = s["case"]
    if case["op"] == "gemm":
        return _grouped_product(s).bfloat16()
    if case["op"] == "gated":
        h = _grouped_product(s)
        gate, up = h[:, :case["I"]], h[:, case["I"]:]
        q, scale = _quantize(gate / (1.0 + torch.exp(-gate)) * up)
        return [q, scale] + ([h.bfloat16()] if case["save"] else [])
    if case["op"] == "gated_backward":
        gate, up = s["h"].float().chunk(2, 1)
        da = s["da"].float()
        sig = 1.0 / (1.0 + torch.exp(-gate))
        dh = torch.cat([da * up * sig * (1.0 + gate * (1.0 - sig)), da * gate * sig], 1)
        return list(_quantize(dh)) if case["fp8"] else [dh.bfloat16()]
    T, top, H = case["T"], case["top"], case["H"]
    rows = s["rows"][s["tok2row"].long()].view(T, top, H).float()
    if case["op"] == "dispatch_backward":
        return rows.sum(1).bfloat16()
    dout = s["dout"].float()
    dw = (rows * dout[:, None]).sum(2)
    dlogits = torch.zeros((T, case["E"]), device=dw.device)
    dlogits.scatter_(1, s["idx"].long(), s["w"] * (dw - (s["w"] * dw).sum(1, keepdim=True)))
    dy = torch.empty((T * top, H), device=dw.device)
    dy[s["tok2row"].long()] = (s["w"][:, :, None] * dout[:, None]).view(T * top, H)
    if case["fp8"]:
        q, scale = _quantize(dy)
        return [q, dw, dlogits, scale]
    return [dy.bfloat16(), dw, dlogits]


# --------------------------------------------------------------------------- its work

def _experts_hit(case):
    """Expected number of experts with a row, and so of weights read."""
    E, T, top = case["E"], case["T"], case["top"]
    p = [(1.0 + e) ** -case.get("zipf", 0.0) for e in range(E)]
    return sum(1.0 - (1.0 - min(1.0, top * v / sum(p))) ** T for v in p)


def work(case):
    op = case["op"]
    if op in ("gemm", "gated"):
        rows, C = case["T"] * case["top"], case["C"]
        N = case["N"] if op == "gemm" else 2 * case["I"]
        b = rows * (C + 4 * _blocks(C)) + _experts_hit(case) * (N * C + 4 * _blocks(N) * _blocks(C))
        if op == "gemm":
            b += rows * N * 2
        else:
            b += rows * (case["I"] + case["I"] // 32) + (rows * N * 2 if case["save"] else 0)
        return {"bytes": b, "flops": 2.0 * rows * N * C}
    if op == "gated_backward":
        rows, inner = case["rows"], case["I"]
        return {"bytes": rows * (6 * inner + (2 * inner + inner // 16 if case["fp8"] else 4 * inner)),
                "flops": 20.0 * rows * inner}
    T, top, H = case["T"], case["top"], case["H"]
    if op == "dispatch_backward":
        return {"bytes": T * top * (H * 2 + 4) + T * H * 2, "flops": T * top * H}
    b = T * H * 2 + T * top * (H * 2 + 16) + T * case["E"] * 4
    b += T * top * (H + H // 32 if case["fp8"] else H * 2)
    return {"bytes": b, "flops": 4.0 * T * top * H}


# --------------------------------------------------------------------------- in 64 bits

def _e4m3_64(v):
    """float64 [n, C], C a multiple of 128: the quantised values (float64) and their scales."""
    n, C = v.shape
    blocks = v.reshape(n, C // 128, 128)
    amax = blocks.abs().max(dim=2).values
    amax = torch.maximum(amax, torch.full_like(amax, AMAX_FLOOR))
    z = blocks * (E4M3_MAX / amax)[:, :, None]
    # the grid of e4m3: 3 bits below the leading one, steps of 2^-9 under 2^-6
    step = torch.exp2(torch.floor(torch.log2(z.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(z / step) * step).clamp(-E4M3_MAX, E4M3_MAX).reshape(n, C), amax / E4M3_MAX


def exact(case, seed):
    op = case["op"]
    if work(case)["flops"] > 1e13:
        return None
    s = prepare(case, seed)
    if op in ("gemm", "gated"):
        a, w = s["a"], s["w"]
        bound = s["offsets"].tolist()
        parts = []
        for e in range(case["E"]):
            lo, hi = bound[e], bound[e + 1]
            if lo == hi:
                continue
            ae, we = a[lo:hi].double(), w[e].double()
            for b in range(_blocks(ae.shape[1])):
                ae[:, 128 * b:128 * b + 128] *= s["a_scale"][lo:hi, b:b + 1].double()
            scale = s["w_scale"][e].double()[torch.arange(we.shape[0], device=we.device) // 128]
            we *= scale[:, torch.arange(we.shape[1], device=we.device) // 128]
            parts.append(ae @ we if case.get("transpose") else ae @ we.T)
        h = torch.cat(parts)
        if op == "gemm":
            return h
        gate, up = h[:, :case["I"]], h[:, case["I"]:]
        q, scale = _e4m3_64(gate * torch.sigmoid(gate) * up)
        return [q, scale] + ([h] if case["save"] else [])
    if op == "gated_backward":
        inner = case["I"]
        gate, up, da = s["h"][:, :inner].double(), s["h"][:, inner:].double(), s["da"].double()
        sig = torch.sigmoid(gate)
        dh = torch.cat([da * up * (sig + gate * sig * (1 - sig)), da * gate * sig], dim=1)
        return list(_e4m3_64(dh)) if case["fp8"] else [dh]
    T, top, H = case["T"], case["top"], case["H"]
    at = s["tok2row"].long().reshape(T, top)
    if op == "dispatch_backward":
        dx = torch.zeros((T, H), dtype=torch.float64, device=at.device)
        for j in range(top):
            dx += s["rows"][at[:, j]].double()
        return dx
    dout, w = s["dout"].double(), s["w"].double()
    dw = torch.stack([(s["rows"][at[:, j]].double() * dout).sum(dim=1) for j in range(top)], dim=1)
    mean = (w * dw).sum(dim=1)
    dlogits = torch.zeros((T, case["E"]), dtype=torch.float64, device=at.device)
    dy = torch.empty((T * top, H), dtype=torch.float64, device=at.device)
    for j in range(top):
        dlogits[torch.arange(T, device=at.device), s["idx"][:, j].long()] = w[:, j] * (dw[:, j] - mean)
        dy[at[:, j]] = w[:, j:j + 1] * dout
    if case["fp8"]:
        q, scale = _e4m3_64(dy)
        return [q, dw, dlogits, scale]
    return [dy, dw, dlogits]
