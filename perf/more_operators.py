"""Cases, plain forms and calls of the operators around a layer of 4-bit experts, for timing and comparison.

Five operators:

* ``rms_norm``: the residual's addition and the root-mean-square norm in front of a layer, the normed
  rows in bf16 and, where wanted, also in e4m3 with one fp32 scale per 128 channels.
* ``rms_norm_backward``: its gradient, to the input (with the residual stream's own gradient added)
  and to the weight.
* ``mx4``: rows to 4-bit floating point (e2m1 values, one power-of-two scale per 32 channels) and back.
* ``gemm``: the experts' product of such rows and weights, over the rows dispatch leaves grouped by
  expert.
* ``gated``: the first product of a gated expert with silu(gate) * up and the 4-bit quantisation of its
  result in one pass.

With ``own`` false ``run`` computes an operator from elementary torch operations in 32 bits;
with ``own`` true it calls this package.
"""
import math

import torch

own = False

EPS = 1e-6
E4M3_MAX = 448.0
AMAX_FLOOR = 2.0 ** -119   # the smallest power of two whose 448 / amax is finite in fp32


def listed():
    return [
        # one token of a decode step in front of its layer: the call's own cost
        dict(name="norm_token", op="norm", T=1, H=7168, residual=True, fp8=True),
        # a decode batch of a narrow model, an odd number of tokens, no residual yet (the first layer)
        dict(name="norm_first_layer", op="norm", T=1003, H=2880, residual=False, fp8=False),
        # the prefill layer: 4096 tokens on each of 8 ranks, bf16 for the router and e4m3 for a shared expert
        dict(name="norm_prefill", op="norm", T=32768, H=7168, residual=True, fp8=True),
        # the toy layer's gradient, where the call's own cost counts
        dict(name="norm_backward_toy", op="norm_backward", T=259, H=256, residual=True),
        # the prefill layer's gradient
        dict(name="norm_backward_prefill", op="norm_backward", T=32768, H=7168, residual=True),
        # the rows a decode batch of 1003 tokens dispatches to its experts, to 4 bits and back
        dict(name="mx4_decode", op="mx4", rows=8024, C=7168),
        # a quarter of the prefill layer's dispatched rows
        dict(name="mx4_prefill", op="mx4", rows=65536, C=7168),
        # one token of a decode step: its 8 experts' second product, bound by reading 8 weights
        dict(name="gemm_token", op="gemm", T=1, E=256, top=8, N=7168, C=2048, zipf=0.0),
        # a decode step with skewed expert load (some experts idle, one with many rows)
        dict(name="gemm_skewed_decode", op="gemm", T=1003, E=384, top=8, N=7168, C=2048, zipf=1.2),
        # the second product of the prefill layer
        dict(name="gemm_prefill", op="gemm", T=32768, E=256, top=8, N=7168, C=2048, zipf=0.0),
        # one token's gated first product
        dict(name="gated_token", op="gated", T=1, E=256, top=8, I=2048, C=7168, zipf=0.0),
        # the gated first product of the prefill layer
        dict(name="gated_prefill", op="gated", T=32768, E=256, top=8, I=2048, C=7168, zipf=0.0),
    ]


_WIDE = (256, 512, 640, 1152, 1664, 2048, 2432, 4096, 5120, 7168)     # multiples of 128
_RAGGED = (208, 400, 720, 1328, 2000, 2880, 4240)                     # multiples of 16 only
_NARROW = (8, 40, 264, 1000, 2888, 16384)                             # of 8
_BLOCKS = (160, 416, 736, 2016, 2880, 4256)                           # of 32 only: whole blocks of 4-bit values


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_backward", "mx4", "gemm", "gemm", "gated"])
    if op == "norm":
        fp8 = rng.random() < 0.5
        H = rng.choice(_WIDE if fp8 else _WIDE + _RAGGED + _NARROW)
        return dict(op=op, T=_log_int(rng, 1, 14000) | 1, H=H, residual=rng.random() < 0.7, fp8=fp8)
    if op == "norm_backward":
        return dict(op=op, T=_log_int(rng, 1, 14000) | 1, H=rng.choice(_WIDE + _RAGGED + _NARROW),
                    residual=rng.random() < 0.7)
    if op == "mx4":
        return dict(op=op, rows=_log_int(rng, 1, 65535) | 1, C=rng.choice(_WIDE + _BLOCKS))
    E = rng.choice([1, 8, 16, 32, 64, 128, 256])
    top = min(E, rng.choice([1, 2, 3, 4, 6, 8]))
    zipf = rng.choice([0.0, 0.0, 0.0, 0.7, 1.2])
    T = _log_int(rng, 1, 2048 if zipf else 32768) | 1
    if op == "gemm":
        N, C = rng.choice(_WIDE + _RAGGED), rng.choice(_WIDE + _BLOCKS)
        case = dict(op=op, T=T, E=E, top=top, N=N, C=C, zipf=zipf)
    else:
        case = dict(op=op, T=T, E=E, top=top, I=rng.choice(_WIDE[:6] + _BLOCKS), C=rng.choice(_WIDE + _BLOCKS), zipf=zipf)
        N, C = 2 * case["I"], case["C"]
    while 2.0 * case["T"] * top * N * C > 4e12 or E * (4.0 * case["T"] * top / E + 64) * C * 4 > 2e10:
        case["T"] = (case["T"] // 2) | 1
    return case


# --------------------------------------------------------------------------- inputs

def _route(case, gen, dev):
    """The rows' bounds by expert for the top experts of normal logits, and each row's token."""
    T, E, top = case["T"], case["E"], case["top"]
    logits = torch.randn((T, E), generator=gen, device=dev)
    if case["zipf"]:   # the log of a Zipf weight over a random order of the experts
        order = torch.randperm(E, generator=gen, device=dev).float()
        logits = logits - case["zipf"] * torch.log1p(order)
    idx = torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :top].reshape(-1)
    offsets = torch.zeros(E + 1, dtype=torch.int64, device=dev)
    offsets[1:] = torch.cumsum(torch.bincount(idx, minlength=E), 0)
    return offsets, torch.sort(idx, stable=True).indices // top


def _power(e):
    """2^e as fp32 for whole numbers in -127..127, exactly (2^-127 is subnormal)."""
    return ((e.int() + 127) << 23).clamp(min=1 << 22).view(torch.float32)


def _mx4(v):
    """fp32 [..., C] -> its e2m1 values (fp32) and the scales' bytes (exponent + 127), one per 32 channels:
    the exponent of the largest magnitude less 2, ties to the even code, 6 where it would be more."""
    blocks = v.unflatten(-1, (-1, 32))
    amax = blocks.abs().amax(-1)
    e = torch.where(amax > 0, torch.frexp(amax).exponent - 3, -127).clamp(min=-127)
    z = blocks * _power(-e)[..., None]
    a = z.abs().clamp(max=6.0)
    step = 0.5 * (1 + (a >= 2) + 2 * (a >= 4))
    return torch.copysign(torch.round(a / step) * step, z).flatten(-2), (e + 127).to(torch.uint8)


def _pack(values):
    """e2m1 values to bytes, the first of a pair in the low half."""
    a = values.abs()
    code = torch.where(a < 2, 2 * a, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    code += (torch.signbit(values).to(torch.uint8) << 3)
    return code[..., 0::2] | (code[..., 1::2] << 4)


def _unpack(q):
    """Bytes to their fp32 values."""
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0],
                         device=q.device)
    return torch.stack([table[(q & 15).int()], table[(q >> 4).int()]], -1).flatten(-2)


def _quantized(shape, gen, dev, gated_values=False):
    """Normal values in 4 bits, some at a time: packed codes and scale bytes.  ``gated_values``: as a
    gated product leaves them."""
    n, C = math.prod(shape[:-1]), shape[-1]
    q = torch.empty((n, C // 2), dtype=torch.uint8, device=dev)
    scale = torch.empty((n, C // 32), dtype=torch.uint8, device=dev)
    most = max(1, (1 << 28) // C)
    for r in range(0, n, most):
        v = torch.randn((min(most, n - r), C), generator=gen, device=dev)
        if gated_values:
            v = torch.nn.functional.silu(v) * torch.randn(v.shape, generator=gen, device=dev)
        else:
            v = v * (1.0 / math.sqrt(C))
        values, s = _mx4(v)
        q[r:r + most], scale[r:r + most] = _pack(values), s
    return q.view(*shape[:-1], C // 2), scale.view(*shape[:-1], C // 32)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    s = dict(case=case)
    op = case["op"]
    if op in ("norm", "norm_backward"):
        T, H = case["T"], case["H"]

        def rows(size):
            return torch.randn((T, H), generator=gen, device=dev).mul_(size).bfloat16()

        s["weight"] = (1.0 + 0.1 * torch.randn(H, generator=gen, device=dev)).bfloat16()
        if op == "norm":
            s["x"], s["y"] = rows(1.0), torch.empty((T, H), dtype=torch.bfloat16, device=dev)
            s["residual"] = rows(3.0) if case["residual"] else None
            s["h"] = torch.empty_like(s["x"]) if case["residual"] else None
            s["q"] = torch.empty((T, H), dtype=torch.float8_e4m3fn, device=dev) if case["fp8"] else None
            s["q_scale"] = torch.empty((T, H // 128), device=dev) if case["fp8"] else None
        else:
            s["h"], s["dy"] = rows(3.0), rows(1e-3)
            s["dh"] = rows(1e-3) if case["residual"] else None
            s["dx"], s["dweight"] = torch.empty_like(s["h"]), torch.empty(H, device=dev)
        return s
    if op == "mx4":
        rows, C = case["rows"], case["C"]
        s["x"] = torch.randn((rows, C), generator=gen, device=dev, dtype=torch.bfloat16)
        s["q"] = torch.empty((rows, C // 2), dtype=torch.uint8, device=dev)
        s["q_scale"] = torch.empty((rows, C // 32), dtype=torch.uint8, device=dev)
        s["out"] = torch.empty_like(s["x"])
        return s
    E, C = case["E"], case["C"]
    N = case["N"] if op == "gemm" else 2 * case["I"]
    offsets, token = _route(case, gen, dev)
    rows = token.numel()
    if op == "gemm":    # the second product has rows of its own
        s["a"], s["a_scale"] = _quantized((rows, C), gen, dev, gated_values=True)
        s["out"] = torch.empty((rows, N), dtype=torch.bfloat16, device=dev)
    else:               # the copies of a token are the same row
        values, scale = _mx4(torch.randn((case["T"], C), generator=gen, device=dev))
        s["a"], s["a_scale"] = _pack(values)[token], scale[token]
        s["q"] = torch.empty((rows, case["I"] // 2), dtype=torch.uint8, device=dev)
        s["q_scale"] = torch.empty((rows, case["I"] // 32), dtype=torch.uint8, device=dev)
        s["values"] = torch.empty((rows, case["I"]), dtype=torch.float8_e4m3fn, device=dev)
    s["w"], s["w_scale"] = _quantized((E, N, C), gen, dev)
    # the experts that have any rows, and the fullest one's count
    counts = torch.diff(offsets)
    s["offsets"], s["hit"], s["most"] = offsets.int(), torch.nonzero(counts).view(-1), int(counts.max())
    return s


# --------------------------------------------------------------------------- one pass

def run(state):
    return _own(state) if own else _plain(state)


def _own(s):
    import combine_moe_route_gb300 as moe
    case = s["case"]
    if case["op"] == "norm":
        r = moe.rms_norm(s["x"], s["weight"], residual=s["residual"], eps=EPS, fp8=case["fp8"], out=s["y"],
                         out_h=s["h"], out_q=s["q"], out_scale=s["q_scale"])
        return [r.y] + ([r.h] if case["residual"] else []) + ([r.q, r.scale] if case["fp8"] else [])
    if case["op"] == "norm_backward":
        r = moe.rms_norm_backward(s["dy"], s["h"], s["weight"], dh=s["dh"], eps=EPS, out=s["dx"],
                                  dweight=s["dweight"])
        return [r.dx, r.dweight]
    if case["op"] == "mx4":
        q, scale = moe.quantize_mx4(s["x"], out=s["q"], out_scale=s["q_scale"])
        return moe.dequantize_mx4(q, scale, out=s["out"])
    if case["op"] == "gemm":
        return moe.expert_gemm_mx4(s["a"], s["a_scale"], s["w"], s["w_scale"], s["offsets"], out=s["out"])
    r = moe.expert_gated_gemm_mx4(s["a"], s["a_scale"], s["w"], s["w_scale"], s["offsets"], out=s["q"],
                                  out_scale=s["q_scale"])
    return [moe.dequantize_mx4(r.q, None, out=s["values"]), r.scale.view(torch.float8_e8m0fnu)]


def _grouped_product(s):
    """fp32 rows of each expert times its weight: experts padded to the fullest, one batched product."""
    rows, dev = s["a"].shape[0], s["a"].device
    hit, most = s["hit"], s["most"]
    first, end = s["offsets"].long()[hit], s["offsets"].long()[hit + 1]
    a = _values(s["a"], s["a_scale"])
    w = _values(s["w"][hit], s["w_scale"][hit])
    padded = a[(first[:, None] + torch.arange(most, device=dev)).clamp(max=rows - 1)]
    out = torch.bmm(padded, w.transpose(1, 2))
    row = torch.arange(rows, device=dev)
    e = torch.searchsorted(end, row, right=True)
    return out.view(hit.numel() * most, -1)[e * most + row - first[e]]


def _values(q, scale):
    """The fp32 values that packed codes and their scales' bytes stand for."""
    v = _unpack(q)
    v.unflatten(-1, (-1, 32)).mul_(_power(scale.int() - 127)[..., None])
    return v


def _quantize_e4m3(v):
    """fp32 [n, C] -> e4m3 [n, C] and fp32 scales [n, C / 128], the rule of the dispatch."""
    blocks = v.unflatten(1, (-1, 128))
    amax = blocks.abs().amax(2).clamp(min=AMAX_FLOOR)
    q = (blocks * (E4M3_MAX / amax)[:, :, None]).clamp(-E4M3_MAX, E4M3_MAX)
    return q.flatten(1).to(torch.float8_e4m3fn), amax / E4M3_MAX


def _plain(s):
    case = s["case"]
    if case["op"] == "norm":
        h = s["x"].float()
        if case["residual"]:
            h = h + s["residual"].float()
        y = h * torch.rsqrt(h.square().mean(1, keepdim=True) + EPS) * s["weight"].float()
        out = [y.bfloat16()] + ([h.bfloat16()] if case["residual"] else [])
        return out + (list(_quantize_e4m3(y)) if case["fp8"] else [])
    if case["op"] == "norm_backward":
        h, dy = s["h"].float(), s["dy"].float()
        r = torch.rsqrt(h.square().mean(1, keepdim=True) + EPS)
        n, g = h * r, dy * s["weight"].float()
        dx = r * (g - n * (g * n).mean(1, keepdim=True))
        if case["residual"]:
            dx = dx + s["dh"].float()
        return [dx.bfloat16(), (dy * n).sum(0)]
    if case["op"] == "mx4":
        values, scale = _mx4(s["x"].float())
        return (values.unflatten(-1, (-1, 32)) * _power(scale.int() - 127)[..., None]).flatten(-2).bfloat16()
    h = _grouped_product(s)
    if case["op"] == "gemm":
        return h.bfloat16()
    gate, up = h[:, :case["I"]], h[:, case["I"]:]
    values, scale = _mx4(gate / (1.0 + torch.exp(-gate)) * up)
    return [values.to(torch.float8_e4m3fn), scale.view(torch.float8_e8m0fnu)]


# --------------------------------------------------------------------------- its work

def _experts_hit(case):
    """About how many experts have a row, and so how many weights are read: a token takes an expert whose
    normal logit, shifted by its load, is over the border that ``top`` of them pass on average."""
    shift = [case["zipf"] * math.log1p(e) for e in range(case["E"])]

    def taken(border):
        return [0.5 * math.erfc((border + s) / math.sqrt(2.0)) for s in shift]

    low, high = -40.0, 40.0
    for _ in range(50):
        middle = (low + high) / 2
        low, high = (middle, high) if sum(taken(middle)) > case["top"] else (low, middle)
    return sum(1.0 - (1.0 - p) ** case["T"] for p in taken(low))


def work(case):
    op = case["op"]
    if op == "norm":
        T, H = case["T"], case["H"]
        b = T * H * (8 if case["residual"] else 4) + 2 * H + (T * (H + H // 32) if case["fp8"] else 0)
        return {"bytes": b, "flops": 6.0 * T * H}
    if op == "norm_backward":
        T, H = case["T"], case["H"]
        return {"bytes": T * H * (8 if case["residual"] else 6) + 6 * H, "flops": 12.0 * T * H}
    if op == "mx4":   # there and back: the 4-bit form is written and read
        n = case["rows"] * case["C"]
        return {"bytes": 4 * n + 2 * (n // 2 + n // 32), "flops": 6.0 * n}
    rows, C = case["T"] * case["top"], case["C"]
    N = case["N"] if op == "gemm" else 2 * case["I"]
    row = C // 2 + C // 32
    b = rows * row + _experts_hit(case) * N * row
    b += rows * N * 2 if op == "gemm" else rows * (case["I"] // 2 + case["I"] // 32)
    return {"bytes": b, "flops": 2.0 * rows * N * C}


# --------------------------------------------------------------------------- in 64 bits

_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _read64(q, scale):
    """float64 values of packed codes [n, C / 2] and scale bytes [n, C / 32]."""
    table = torch.tensor(_E2M1 + tuple(-v for v in _E2M1), dtype=torch.float64, device=q.device)
    v = torch.empty((q.shape[0], 2 * q.shape[1]), dtype=torch.float64, device=q.device)
    v[:, 0::2], v[:, 1::2] = table[(q % 16).long()], table[(q // 16).long()]
    return v * torch.exp2(scale.double() - 127).repeat_interleave(32, dim=1)


def _mx4_64(v):
    """float64 [n, C]: the e2m1 values nearest to the scaled ones, and the scales."""
    n, C = v.shape
    amax = v.abs().reshape(n, C // 32, 32).max(dim=2).values
    # the largest power of two up to amax, then a quarter of it; log2 may round up just below a power
    e = torch.floor(torch.log2(amax.clamp(min=2.0 ** -125)))
    e = torch.where(torch.exp2(e) > amax.clamp(min=2.0 ** -125), e - 1, e)
    scale = torch.where(amax > 0, torch.exp2(e - 2), torch.full_like(e, 2.0 ** -127))
    z = v / scale.repeat_interleave(32, dim=1)
    a, code = z.abs(), torch.zeros_like(z, dtype=torch.int64)
    for i in range(7):   # past the middle between neighbours, or on it where the upper code is even
        middle = (_E2M1[i] + _E2M1[i + 1]) / 2
        code += (a > middle) | ((a == middle) & (i % 2 == 1))
    return torch.tensor(_E2M1, dtype=torch.float64, device=v.device)[code] * torch.sign(z), scale


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
    if op == "norm":
        h, w = s["x"].double(), s["weight"].double()
        if case["residual"]:
            h += s["residual"].double()
        y = h / torch.sqrt((h * h).sum(dim=1) / case["H"] + EPS)[:, None] * w
        out = [y] + ([h] if case["residual"] else [])
        return out + (list(_e4m3_64(y)) if case["fp8"] else [])
    if op == "norm_backward":
        h, dy, w, H = s["h"].double(), s["dy"].double(), s["weight"].double(), case["H"]
        size = torch.sqrt((h * h).sum(dim=1) / H + EPS)[:, None]
        dx = dy * w / size - h * (dy * w * h).sum(dim=1)[:, None] / (H * size ** 3)
        if case["residual"]:
            dx += s["dh"].double()
        return [dx, torch.einsum("th,th->h", dy, h / size)]
    if op == "mx4":
        out = torch.empty((case["rows"], case["C"]), dtype=torch.float64, device=s["x"].device)
        for r in range(0, case["rows"], 16384):
            values, scale = _mx4_64(s["x"][r:r + 16384].double())
            out[r:r + 16384] = values * scale.repeat_interleave(32, dim=1)
        return out
    bound, parts = s["offsets"].tolist(), []
    for e in range(case["E"]):
        if bound[e] < bound[e + 1]:
            rows = slice(bound[e], bound[e + 1])
            h = _read64(s["a"][rows], s["a_scale"][rows]) @ _read64(s["w"][e], s["w_scale"][e]).T
            parts.append(h if op == "gemm" else _mx4_64(h[:, :case["I"]] * torch.sigmoid(h[:, :case["I"]])
                                                        * h[:, case["I"]:]))
    if op == "gemm":
        return torch.cat(parts)
    return [torch.cat([p[0] for p in parts]), torch.cat([p[1] for p in parts])]
