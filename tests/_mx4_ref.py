"""64-bit references of the 4-bit rows and their products (CPU, torch), and what the tests allow."""
import numpy as np
import torch

LEVELS = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)


def scale_byte(amax):
    """The scale bytes of blocks with these largest magnitudes (float64, finite)."""
    e = torch.frexp(amax).exponent.long() - 1
    return torch.where(amax > 0, (e - 2 + 127).clamp(min=0), torch.zeros_like(e))


def quantize(v):
    """float64 [..., C] -> codes uint8 [..., C] (one a byte) and scale bytes uint8 [..., C/32]."""
    b = v.unflatten(-1, (-1, 32))
    bad = ~torch.isfinite(b).all(-1)
    b = torch.where(bad[..., None], torch.zeros_like(b), b)
    byte = scale_byte(b.abs().amax(-1))
    z = b * torch.exp2(127.0 - byte.double())[..., None]
    a, code = z.abs(), torch.zeros(z.shape, dtype=torch.long)
    for i in range(7):
        middle = (LEVELS[i] + LEVELS[i + 1]) / 2
        code += (a > middle) | ((a == middle) & (i % 2 == 1))
    code += 8 * torch.signbit(z).long()
    code[bad] = 0
    byte[bad] = 255
    return code.flatten(-2).to(torch.uint8), byte.to(torch.uint8)


def pack(codes):
    return codes[..., 0::2] | (codes[..., 1::2] << 4)


def unpack(q):
    return torch.stack([q & 15, q >> 4], -1).flatten(-2)


def code_values(codes):
    v = LEVELS[(codes & 7).long()]
    return torch.where(codes >= 8, -v, v)


def scale_values(byte):
    s = torch.exp2(byte.double() - 127.0)
    s[byte == 255] = float("nan")
    return s


def values(q, byte):
    """The float64 values of packed codes and scale bytes."""
    return (code_values(unpack(q)).unflatten(-1, (-1, 32)) * scale_values(byte)[..., None]).flatten(-2)


def random_rows(shape, rng, spread=3):
    """Random codes (all sixteen) and scales of 2^(-spread..spread)."""
    q = torch.from_numpy(rng.integers(0, 256, (*shape[:-1], shape[-1] // 2), dtype=np.uint8))
    s = torch.from_numpy(rng.integers(127 - spread, 128 + spread, (*shape[:-1], shape[-1] // 32), dtype=np.uint8))
    return q, s


def product_inputs(counts, N, C, rng, spread=3):
    E, rows = len(counts), int(sum(counts))
    off = np.zeros(E + 1, dtype=np.int32)
    off[1:] = np.cumsum(counts)
    a, sa = random_rows((rows, C), rng, spread)
    w, sw = random_rows((E, N, C), rng, spread)
    return dict(a=a, a_scale=sa, w=w, w_scale=sw, off=torch.from_numpy(off))


def product(inp):
    """(result, sum of |terms|) in float64; zeros for rows no expert owns."""
    a, w = values(inp["a"], inp["a_scale"]), values(inp["w"], inp["w_scale"])
    out = torch.zeros((a.shape[0], w.shape[1]), dtype=torch.float64)
    mag = torch.zeros_like(out)
    off = inp["off"].tolist()
    for e in range(w.shape[0]):
        rows = slice(off[e], off[e + 1])
        out[rows] = a[rows] @ w[e].T
        mag[rows] = a[rows].abs() @ w[e].abs().T
    return out, mag


def product_bound(mag, C):
    """Error of an fp32 accumulation of C terms against exact arithmetic.

    Products of two 4-bit values and of two scales are exact.  Per group of 16 terms the running sum
    may lose 2^-22 of the largest magnitude it can reach (mag): one rounding or truncation of the sum
    and one of the group's own; 16 more for the sums of a contraction that blocks share."""
    return (C / 16 + 16) * 2.0 ** -22 * mag


def quantized_ok(q, byte, v, err):
    """Whether (q packed, byte) is the quantisation of values within err of v (float64 [n, C]): the
    scale is that of a largest magnitude within err, every value is within half a step of v (the
    steps below and above a level differ: the larger counts), or 6 with v up to 8."""
    amax, worst = v.abs().unflatten(-1, (-1, 32)).amax(-1), err.unflatten(-1, (-1, 32)).amax(-1)
    low, high = scale_byte((amax - worst).clamp(min=0)), scale_byte(amax + worst)
    ok_scale = ((byte.long() >= low) & (byte.long() <= high)).all()
    s = scale_values(byte).repeat_interleave(32, -1)
    x = code_values(unpack(q))
    a = x.abs()
    half = torch.where(a < 2, 0.25, torch.where(a < 4, 0.5, torch.where(a < 6, 1.0, 2.0)))
    ok_value = ((x * s - v).abs() <= half * s + err).all()
    return bool(ok_scale), bool(ok_value)
