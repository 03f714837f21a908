"""Plain 64-bit forms of the microscaled operators, on the CPU.  Shares nothing with
the CUDA path."""
import torch

E2M1 = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)
E2M1 = torch.cat([E2M1, -E2M1])


def _e4m3():
    v = []
    for c in range(256):
        e, f = (c >> 3) & 15, c & 7
        x = (8 + f) * 2.0 ** (e - 10) if e else f * 2.0 ** -9
        v.append(float("nan") if c & 127 == 127 else -x if c & 128 else x)
    return torch.tensor(v, dtype=torch.float64)


E4M3 = _e4m3()


def unpack4(codes):
    """Code numbers of int32 words, low bits first."""
    c = codes.long() & 0xFFFFFFFF
    return torch.stack([(c >> (4 * i)) & 15 for i in range(8)], -1).flatten(-2)


def pack4(numbers):
    c = (numbers.long().unflatten(-1, (-1, 8)) << (4 * torch.arange(8))).sum(-1)
    return torch.where(c >= 1 << 31, c - (1 << 32), c).int()


def scale_of(scales):
    s = torch.pow(torch.tensor(2.0, dtype=torch.float64), scales.double() - 127)
    return torch.where(scales == 255, float("nan"), s)


def values(codes, scales):
    """float64 values of MXFP4 (int32 codes) or MXFP8 (uint8) rows."""
    v = E2M1[unpack4(codes)] if codes.dtype == torch.int32 else E4M3[codes.long()]
    return v * scale_of(scales).repeat_interleave(32, -1)


def lead(a):
    """floor(log2 a) of positive float64."""
    return torch.frexp(a).exponent - 1


def scale_bytes(x, bits):
    """Scale byte of each block of float64 rows."""
    a = x.unflatten(-1, (-1, 32)).abs().amax(-1)
    odd = ~torch.isfinite(a)
    b = torch.where(a > 0, lead(torch.where(odd | (a == 0), 1.0, a)) - (2 if bits == 4 else 8) + 127, 0)
    return torch.where(odd, 255, b.clamp(min=0)).to(torch.uint8)


def grid_step(v, bits):
    """Step of the code grid around magnitudes v (already divided by the scale)."""
    emin, mant = (0, 1) if bits == 4 else (-6, 3)
    e = lead(torch.where(v > 0, v, 1.0)).double()
    e = torch.where(v > 0, e, float(emin)).clamp(min=emin)
    return torch.pow(2.0, e - mant)


def quantize(x, bits):
    """(code numbers, scale bytes) of float64 rows whose blocks are finite."""
    s = scale_bytes(x, bits)
    v = x / scale_of(s).repeat_interleave(32, -1)
    a = v.abs()
    step = grid_step(a, bits)
    a = torch.clamp(torch.round(a / step) * step, max=6.0 if bits == 4 else 448.0)
    table = E2M1[:8] if bits == 4 else E4M3[:127]
    c = torch.searchsorted(table, a.contiguous())
    return c + torch.signbit(v).long() * (8 if bits == 4 else 128), s


def check_mx8(codes, scales, want, tol, what):
    """MXFP8 rows against float64 rows that are known to within tol: each scale is that of
    some magnitude in reach, each value the nearest code or one no further off than tol."""
    a = want.unflatten(-1, (-1, 32)).abs()
    t = tol.unflatten(-1, (-1, 32)) if isinstance(tol, torch.Tensor) else torch.full_like(a, tol)
    most, reach = a.amax(-1), t.amax(-1)
    s = scales.long()
    lo = torch.where(most > reach, (lead((most - reach).clamp(min=2.0 ** -400)) - 8 + 127).clamp(min=0), 0)
    hi = torch.where(most + reach > 0, (lead((most + reach).clamp(min=2.0 ** -400)) - 8 + 127).clamp(min=0), 0)
    bad = (s < lo) | (s > hi)
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} scales, first {s[bad][:4]} {lo[bad][:4]} {hi[bad][:4]}"
    got = values(codes, scales)
    unit = scale_of(scales).repeat_interleave(32, -1)
    tt = t.flatten(-2)
    size = (want.abs() + tt) / unit
    most_off = 0.5 * grid_step(torch.maximum(size, got.abs() / unit), 8) * unit + tt
    # above the largest code: the scale was chosen so that the value was below 512 of it
    cut = (got.abs() / unit == 448) & (want.abs() + tt >= got.abs()) & ((want.abs() - tt) / unit < 512)
    off = (got - want).abs()
    wrong = ~((off <= most_off) | (cut & (got.sign() == want.sign())))
    assert not bool(wrong.any()), (f"{what}: {int(wrong.sum())} of {wrong.numel()} values, first "
                                   f"{got[wrong][:4]} for {want[wrong][:4]}")


def product(w, x):
    """y = x W^T in float64 and how far an fp32 product may be from it: a step of 32
    products is added to the sum so far with an error of at most 2^-20 of both (33 terms,
    aligned to the largest and cut 2^-25 below it)."""
    wv, xv = values(*w), x
    y = xv @ wv.T
    size, part = torch.zeros_like(y), torch.zeros_like(y)
    k = xv.shape[-1]
    for i in range(0, k, 32):
        a, b = xv[:, i:i + 32], wv[:, i:i + 32]
        size += a.abs() @ b.abs().T
        part += a @ b.T
        size += part.abs()
    return y, 2.0 ** -20 * size


# Products (rows of x, rows of weights, K, two weights) that pairs of thread blocks work on: some
# tiles of a block, sizes that no tile divides, K of whole and of parts of the loaders' 512.
PAIRS = [(777, 2051, 1024, 0), (1500, 5000, 256, 0), (2100, 8000, 128, 0), (333, 2500, 1152, 0), (225, 30000, 128, 0),
         (1000, 513, 4096, 0), (1000, 2048, 2048, 1), (300, 1440, 512, 1), (100, 2816, 1024, 1), (3000, 2016, 2048, 1),
         (640, 1001, 896, 1)]
PAIRS_SMALL = [(333, 1001, 640, 0), (333, 1004, 640, 0), (333, 1004, 640, 1), (130, 1952, 896, 1)]
PAIRS_LARGEST, PAIRS_GRAPH = (45050, 50000, 2048), (400, 1504, 1152)


def gated(g, tg, u, tu):
    """silu(g) u and its error for g, u off by tg, tu: |silu'| <= 1.1, |silu(g)| <= |g|;
    expf, the division and the products take a few 2^-24 of the result, 2^-20 in all (and
    2^-22 of g by the exponent, where -g is large and silu small)."""
    s = g * torch.sigmoid(g)
    h = s * u
    return h, 1.1 * tg * (u.abs() + tu) + s.abs() * tu + 2.0 ** -20 * h.abs() + 2.0 ** -140


def near(got, want, tol, what):
    """fp16 outputs: tol and half a step of fp16 (2^-11, 2^-25 below 2^-14)."""
    got = got.double().cpu()
    t = tol + 2.0 ** -11 * (want.abs() + tol) + 2.0 ** -25
    over = want.abs() + t >= 65520
    same = ((got - want).abs() <= t) | (over & (got.abs() >= 65504))
    assert bool(same.all()), (f"{what}: {int((~same).sum())} of {same.numel()} outside, worst "
                              f"{float(((got - want).abs() / t)[~same].max())} x tolerance")
