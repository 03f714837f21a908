"""The microscaled products where their values are extreme, against plain 64-bit forms."""
import pytest
import torch

import mx_reference as ref

pytestmark = pytest.mark.gpu

q = pytest.importorskip("bit_group_quantized_qgemv_gb300")


def dev(pair):
    return tuple(t.cuda() for t in pair)


# (blocks by themselves, clusters that share K, pairs)
@pytest.mark.parametrize("n,k", [(64, 96), (160, 9216), (2816, 1024)])
@pytest.mark.parametrize("sign", [-1, 1])
@pytest.mark.parametrize("up_scale", [127, 140, 250])
def test_gates_far_from_zero(n, k, sign, up_scale):
    """Gates of 60 to 104 on either side times 1, 2^13 and 2^123: results that fp32 holds are there,
    however small their gate is.  Both sums are exact: three products and one."""
    z = torch.arange(60, 104.25, 0.25, dtype=torch.float64)
    parts = torch.stack([z - z % 8, (z % 8).floor(), z % 1], 1)
    codes = torch.searchsorted(ref.E4M3[:127], parts)
    assert torch.equal(ref.E4M3[codes], parts)
    m = len(z)
    x = torch.zeros(m, k, dtype=torch.uint8)
    x[:, [0, 9, 31]] = (codes + (128 if sign < 0 else 0)).to(torch.uint8)
    x[:, 32] = 0x38                                                       # 1
    xs = torch.full((m, k // 32), 127, dtype=torch.uint8)
    gate, up = (torch.zeros(n, k, dtype=torch.long) for _ in range(2))
    gate[:, [0, 9, 31]] = 2
    up[:, 32] = 2
    gs, us = torch.full((n, k // 32), 127, dtype=torch.uint8), torch.full((n, k // 32), up_scale, dtype=torch.uint8)
    h = torch.zeros(m, n, dtype=torch.float16, device="cuda")
    c, s = torch.zeros(m, n, dtype=torch.uint8, device="cuda"), torch.zeros(m, n // 32, dtype=torch.uint8, device="cuda")
    q.mx_swiglu(dev((ref.pack4(gate), gs)), dev((ref.pack4(up), us)), dev((x, xs)), h=h, codes=c, scales=s)
    z, u = sign * z, 2.0 ** (up_scale - 127)
    want = z * torch.sigmoid(z) * u
    # e^-|z|: 2 + 1.18 |z| units in the last place (2^-23), half a unit of the smallest subnormal;
    # z e^z, 1 + e and the product with u half a unit each, the division two
    tol = want.abs() * (2.0 ** -20 + z.abs() * 2.0 ** -22) + z.abs() * 2.0 ** -149 * u
    want, tol = want[:, None].expand(m, n), tol[:, None].expand(m, n)
    ref.near(h, want, tol, "fp16")
    if sign > 0 and up_scale == 250:
        # 60 * 2^123 = 1.9 * 2^128 and more: no fp32 value, an infinity, whose blocks are NaN
        assert float(want.min()) > 2.0 ** 128 and bool((s == 255).all()) and bool(torch.isinf(h).all())
        return
    ref.check_mx8(c.cpu(), s.cpu(), want, tol, "MXFP8")
    assert q.device_status() == 0


def test_scales_of_another_shape_are_refused():
    """As many scales as there are blocks, but in a transposed matrix or a flat array; weights in a stack."""
    n, m, k = 96, 6, 128
    x = torch.ones(m, k, dtype=torch.float16, device="cuda")
    codes, scales = q.mx_quantize(torch.ones(n, k, dtype=torch.float16, device="cuda"), 4)
    xc, xs = q.mx_quantize(x)
    c4, s4 = q.mx_quantize(x, 4)
    w, gamma = (codes, scales), torch.ones(k, dtype=torch.float16, device="cuda")
    y = torch.zeros(m, n, dtype=torch.float16, device="cuda")
    for wrong in (lambda t: t.t().contiguous(), lambda t: t.flatten(), lambda t: t.unsqueeze(-1)):
        for call in (lambda: q.mx_quantize(x, 8, scales=wrong(xs)), lambda: q.mx_quantize(x, 4, scales=wrong(s4)),
                     lambda: q.mx_dequantize(xc, wrong(xs)), lambda: q.mx_dequantize(c4, wrong(s4)),
                     lambda: q.residual_rmsnorm_mxfp8(x, gamma, scales=wrong(xs)),
                     lambda: q.qgemv_mxfp4((codes, wrong(scales)), x), lambda: q.mx_gemm((codes, wrong(scales)), (xc, xs)),
                     lambda: q.mx_gemm(w, (xc, wrong(xs))), lambda: q.mx_swiglu((codes, wrong(scales)), w, (xc, xs)),
                     lambda: q.mx_swiglu(w, (codes, wrong(scales)), (xc, xs)), lambda: q.mx_swiglu(w, w, (xc, wrong(xs))),
                     lambda: q.mx_swiglu(w, w, (xc, xs), scales=wrong(torch.zeros(m, n // 32, dtype=torch.uint8, device="cuda")))):
            with pytest.raises(ValueError):
                call()
    stack = (codes.view(4, 24, k // 8), scales.view(4, 24, k // 32))
    for call in (lambda: q.qgemv_mxfp4(stack, x, y=y), lambda: q.mx_gemm(stack, (xc, xs), y=y),
                 lambda: q.mx_swiglu(stack, w, (xc, xs), h=y), lambda: q.mx_swiglu(w, stack, (xc, xs), h=y)):
        with pytest.raises(ValueError):
            call()
    assert q.mx_gemm(w, (xc, xs), y=y) is y


@pytest.mark.parametrize("top", [65504.0, 33000.0, 4000.0, 511.75, 256.0, 255.875, 16.0, 7.5, 1.0, 2.0 ** -9, 2.0 ** -16, 2.0 ** -23])
def test_every_fp16_value_beside_a_larger_one(top):
    """Every fp16 value up to the largest one of its block, in rows of one to eight: exact where that
    is below 32768; beside larger ones fp16's last place, 2^-24, is rounded to a multiple of 2^-23."""
    every = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16).view(torch.float16)
    every = every[torch.isfinite(every) & (every.abs().float() <= top)]
    k = 1024                                                   # 32 blocks of 31 values and the largest
    per = 31 * 32
    rows = -(-every.numel() // per)
    x = torch.zeros(rows * per, dtype=torch.float16)
    x[:every.numel()] = every[torch.randperm(every.numel(), generator=torch.Generator().manual_seed(1))]
    x = torch.cat([torch.full((rows, 32, 1), top, dtype=torch.float16), x.view(rows, 32, 31)], 2).view(rows, k)
    one = torch.zeros(k, k, dtype=torch.long)
    one[torch.arange(k), torch.arange(k)] = 2
    w = dev((ref.pack4(one), torch.full((k, k // 32), 127, dtype=torch.uint8)))
    got, at = [], 0
    while at < rows:                                           # 8, 1, 2, ... rows a call
        n = 8 if at < rows - 20 else 1 + at % 8
        got.append(q.qgemv_mxfp4(w, x[at:at + n].cuda()).cpu())
        at += n
    off = (torch.cat(got).double() - x.double()).abs()
    assert float(off.max()) <= (0.0 if top < 32768 else 2.0 ** -24)


@pytest.mark.parametrize("large,small", [(1000.0, 1e-2), (2000.0, 1e-3), (60000.0, 1e-3), (60000.0, 1e-4), (-60000.0, 3e-6),
                                         (65504.0, 6e-8), (250.0, 6e-8), (1.0, 6e-8)])
@pytest.mark.parametrize("m,n,k", [(1, 40, 32), (5, 300, 1120), (8, 200, 8192)])
def test_small_values_beside_one_without_weight(large, small, m, n, k):
    """The largest value of each block times a weight of 0: nothing of it is in the sum, all of the others is."""
    g = torch.Generator().manual_seed(m)
    x = (small * (1 + torch.rand(m, k, generator=g))).half()
    x.view(m, -1, 32)[:, :, 7] = large
    numbers = torch.randint(0, 8, (n, k), generator=g)
    numbers.view(n, -1, 32)[:, :, 7] = 0
    w = ref.pack4(numbers), torch.full((n, k // 32), 127, dtype=torch.uint8)
    # a value is held exactly beside less than 32768, else in multiples of 2^-23 (three columns of three
    # significant bits and a sign, 2^-24 of the last one's smallest step of 2^-16 being the last place of
    # values halved to below 2^15): half of that off; no product of the large one is there to align others to
    y = x.double().clone()
    y.view(m, -1, 32)[:, :, 7] = 0
    want, tol = ref.product(w, y)
    held = torch.full_like(y, 2.0 ** -24 if abs(large) >= 32768 else 0.0)
    ref.near(q.qgemv_mxfp4(dev(w), x.cuda()), want, tol + held @ ref.values(*w).T, "small values")
    assert q.device_status() == 0
