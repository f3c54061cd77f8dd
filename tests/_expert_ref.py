"""64-bit references of the expert products and the gradients (CPU, numpy and torch), and the
error bounds the tests allow."""
import numpy as np
import torch

AMAX_FLOOR = 2.0 ** -119
E4M3_MAX = 448.0


def blocks(n):
    return -(-n // 128)


def random_e4m3(shape, rng, sigma=100.0):
    v = torch.from_numpy(rng.standard_normal(shape).astype(np.float32) * np.float32(sigma))
    return v.clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)


def random_scales(shape, rng, size=1.0):
    return torch.from_numpy((size * rng.uniform(0.25, 4.0, shape)).astype(np.float32))


def product_inputs(counts, N, C, rng, transpose=False):
    """e4m3 rows and weights with scales, and the offsets of `counts` rows per expert."""
    E, rows = len(counts), int(sum(counts))
    wshape = (E, C, N) if transpose else (E, N, C)
    off = np.zeros(E + 1, dtype=np.int32)
    off[1:] = np.cumsum(counts)
    return dict(a=random_e4m3((rows, C), rng), a_scale=random_scales((rows, blocks(C)), rng, 0.01),
                w=random_e4m3(wshape, rng),
                w_scale=random_scales((E, blocks(wshape[1]), blocks(wshape[2])), rng, 1e-4),
                off=torch.from_numpy(off))


def _dequant_rows(q, scale):
    v = q.double()
    return v * scale.double().repeat_interleave(128, 1)[:, :v.shape[1]]


def _dequant_weight(q, scale):
    v = q.double()
    s = scale.double().repeat_interleave(128, 1)[:, :v.shape[1]].repeat_interleave(128, 2)[:, :, :v.shape[2]]
    return v * s


def product(inp, transpose=False):
    """(result, sum of |terms|) in float64; zeros for rows no expert owns."""
    a, w = _dequant_rows(inp["a"], inp["a_scale"]), _dequant_weight(inp["w"], inp["w_scale"])
    if transpose:
        w = w.transpose(1, 2)
    out = torch.zeros((a.shape[0], w.shape[1]), dtype=torch.float64)
    mag = torch.zeros_like(out)
    off = inp["off"].tolist()
    for e in range(w.shape[0]):
        lo, hi = off[e], off[e + 1]
        out[lo:hi] = a[lo:hi] @ w[e].T
        mag[lo:hi] = a[lo:hi].abs() @ w[e].abs().T
    return out, mag


def product_bound(mag, C):
    """Error of an fp32 contraction of C terms against exact arithmetic.

    Products of two e4m3 values are exact in fp32.  Per group of 16 terms the running sum may
    lose 2^-22 of the largest magnitude it can reach (mag): one rounding or truncation of the
    sum and one of the group's own; the scales add a few roundings more."""
    return (C / 16 + 16) * 2.0 ** -22 * mag


def quantized_ok(q, scale, v, err):
    """Whether (q, scale) is the block quantisation of values within err of v (float64 [n, C],
    C a multiple of 128): the scale is amax / 448 within err / 448 and a few fp32 roundings, and
    every dequantised value is within half an e4m3 step of v."""
    n, C = v.shape
    q, scale = q.double(), scale.double()
    amax = v.abs().view(n, -1, 128).amax(2)
    ref = torch.clamp(amax, min=AMAX_FLOOR) / E4M3_MAX
    worst = err.view(n, -1, 128).amax(2)
    ok_scale = ((scale - ref).abs() <= ref * 2.0 ** -21 + worst / E4M3_MAX).all()
    s = scale.repeat_interleave(128, 1)
    half_step = torch.clamp(q.abs() * 2.0 ** -4, min=2.0 ** -10)   # e4m3: 3 fraction bits, subnormal step 2^-9
    ok_value = ((q * s - v).abs() <= s * half_step * (1 + 2.0 ** -20) + err + v.abs() * 2.0 ** -20).all()
    return bool(ok_scale), bool(ok_value)


def quantize_f32(v):
    """The dispatch's rule on fp32 values, step by step in fp32: e4m3 bytes and scales."""
    n, C = v.shape
    b = v.view(n, C // 128, 128)
    amax = torch.clamp(b.abs().amax(2), min=np.float32(AMAX_FLOOR).item())
    inv = torch.full_like(amax, E4M3_MAX) / amax
    q = (b * inv[:, :, None]).clamp(-E4M3_MAX, E4M3_MAX).view(n, C).to(torch.float8_e4m3fn)
    return q, amax / torch.full_like(amax, E4M3_MAX)


def gate(g, u):
    return g / (1.0 + torch.exp(-g)) * u


def gate_grad(g, u, dv):
    """(dg, du, error bound) of v = silu(g) * u in float64.

    expf is within 2 ulp, and each product, sum and division rounds once: fewer than 16
    roundings of 2^-24 reach a term, each of at most |dv| * (|u| * (1 + |g|) + |g|)."""
    s = torch.sigmoid(g)
    dg, du = dv * u * s * (1 + g * (1 - s)), dv * g * s
    bound = 32 * 2.0 ** -24 * dv.abs() * (u.abs() * (1 + g.abs()) + g.abs())
    return dg, du, bound


def combine_grads(dout, y, tok2row, w, idx, E):
    """(dy fp64 or None where no copy maps, dw, dlogits, bounds of the last two) in float64."""
    T, K = w.shape
    rows, H = y.shape
    at = tok2row.long().view(T, K)
    ok = (at >= 0) & (at < rows)
    take = y.double()[at.clamp(0, max(rows - 1, 0))] if rows else torch.zeros((T, K, H), dtype=torch.float64)
    take = take * ok[:, :, None]
    d, wd = dout.double()[:, None], w.double()
    dw = (take * d).sum(2)
    # an fp32 sum of H products in any order: H roundings of 2^-24 of the terms' magnitudes
    dw_err = H * 2.0 ** -24 * (take * d).abs().sum(2)
    mean = (wd * dw).sum(1, keepdim=True)
    dl = torch.zeros((T, E), dtype=torch.float64).scatter_(1, idx.long(), wd * (dw - mean))
    mag = dw.abs() + (wd * dw.abs()).sum(1, keepdim=True)
    e = wd * (dw_err + (wd * dw_err).sum(1, keepdim=True) + (K + 4) * 2.0 ** -24 * mag)
    dl_err = torch.zeros((T, E), dtype=torch.float64).scatter_(1, idx.long(), e)
    dy = torch.full((rows, H), float("nan"), dtype=torch.float64)
    dy[at[ok]] = (wd[:, :, None] * d)[ok]
    return dy, dw, dl, dw_err, dl_err
