"""The microscaled operators (mx_quantize, mx_dequantize, residual_rmsnorm_mxfp8,
qgemv_mxfp4, mx_gemm, mx_swiglu) against plain 64-bit forms: every code and scale, sizes
that fit no tile, rows from none to many, odd alignments, values that are not finite,
captured graphs, streams, and the operators in a row as a layer uses them."""
import pytest
import torch

import mx_reference as ref

pytestmark = pytest.mark.gpu

q = pytest.importorskip("bit_group_quantized_qgemv_gb300")


def gen(seed):
    return torch.Generator().manual_seed(seed)


def rows16(seed, m, k, scale=1.0):
    """fp16 rows with channels of different sizes."""
    g = gen(seed)
    return (torch.randn(m, k, generator=g) * torch.exp(0.8 * torch.randn(k, generator=g)) * scale).half()


def weight(seed, n, k, spread=3):
    """Random MXFP4 codes, every code and scales of some powers of two."""
    g = gen(seed)
    numbers = torch.randint(0, 16, (n, k), generator=g)
    scales = torch.randint(122 - spread, 122 + spread, (n, k // 32), generator=g).to(torch.uint8)
    return ref.pack4(numbers), scales


def acts(seed, m, k):
    """MXFP8 rows as the quantiser makes them."""
    c, s = ref.quantize(rows16(seed, m, k).double(), 8)
    return c.to(torch.uint8), s


def dev(pair):
    return tuple(t.cuda() for t in pair)


def placed(t, offset):
    """A copy on the GPU that starts `offset` bytes behind a 256-byte boundary."""
    raw = torch.zeros(t.numel() * t.element_size() + 256, dtype=torch.uint8, device="cuda")
    out = raw[offset:offset + t.numel() * t.element_size()].view(t.dtype).view(t.shape)
    out.copy_(t)
    assert out.data_ptr() % 256 == offset
    return out


# ------------------------------------------------------------- quantisation

@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("m,k", [(1, 32), (1, 64), (3, 96), (17, 1120), (130, 4096), (1, 16384), (2049, 32)])
def test_quantize(bits, m, k):
    x = rows16(m * 7 + k, m, k)
    x[0, :32] = 0
    x[-1, -32:] *= 0.0                                      # zeros of both signs
    c, s = q.mx_quantize(x.cuda(), bits)
    want, ws = ref.quantize(x.double(), bits)
    got = ref.unpack4(c.cpu()) if bits == 4 else c.cpu().long()
    assert torch.equal(s.cpu(), ws)
    assert torch.equal(got, want)
    v = q.mx_dequantize(c, s)
    assert torch.equal(v.cpu().double(), ref.values(c.cpu(), s.cpu()))


@pytest.mark.parametrize("bits", [4, 8])
def test_quantize_every_fp16(bits):
    """Every finite fp16 value, beside a largest one of every exponent."""
    all16 = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16).view(torch.float16)
    all16 = all16[torch.isfinite(all16)]
    all16 = all16[torch.argsort(all16.abs().float(), stable=True)]
    x = all16[:all16.numel() // 31 * 31].view(-1, 31)
    tops = x[:, -1:].abs()
    more = torch.cat([torch.cat([x, tops * f], 1) for f in (1.0, 1.5, 2.0, 8.0, 256.0, 4096.0)])
    more = more[torch.isfinite(more).all(1)]
    c, s = q.mx_quantize(more.cuda(), bits)
    want, ws = ref.quantize(more.double(), bits)
    assert torch.equal(s.cpu(), ws)
    assert torch.equal(ref.unpack4(c.cpu()) if bits == 4 else c.cpu().long(), want)


@pytest.mark.parametrize("bits", [4, 8])
def test_quantize_not_finite(bits):
    x = rows16(3, 4, 128)
    x[0, 5], x[1, 40], x[2, 70], x[3, 127] = float("nan"), float("inf"), -float("inf"), -float("nan")
    c, s = q.mx_quantize(x.cuda(), bits)
    _, ws = ref.quantize(torch.nan_to_num(x.double(), 1.0, 1.0, 1.0), bits)
    ws = torch.where(torch.isfinite(x.view(4, 4, 32)).all(-1), ws, 255)
    ok = ws != 255
    assert torch.equal(s.cpu()[ok], ws[ok]) and bool((s.cpu()[~ok] == 255).all())
    v = q.mx_dequantize(c, s).cpu().view(4, 4, 32)
    assert bool(torch.isnan(v[~ok]).all()) and bool(torch.isfinite(v[ok]).all())


@pytest.mark.parametrize("bits", [4, 8])
def test_dequantize_every_code_and_scale(bits):
    n = 16 if bits == 4 else 256
    numbers = torch.arange(n).repeat(256 * 32 // n, 1).view(-1, 32) if n <= 32 else torch.arange(n).view(8, 32).repeat(256, 1)
    scales = torch.arange(256).repeat_interleave(numbers.shape[0] // 256).to(torch.uint8).view(-1, 1)
    codes = ref.pack4(numbers) if bits == 4 else numbers.to(torch.uint8)
    got = q.mx_dequantize(codes.cuda(), scales.cuda()).cpu()
    want = ref.values(codes, scales).half()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(torch.nan_to_num(got, 0, 70000, -70000), torch.nan_to_num(want, 0, 70000, -70000))


# --------------------------------------------------------------------- norm

@pytest.mark.parametrize("m,k,res", [(1, 32, True), (1, 4096, True), (1, 4096, False), (5, 96, True), (3, 160, False),
                                     (9, 256, True), (33, 1120, True), (2, 16384, True), (2, 20000 // 32 * 32, False),
                                     (4, 40960, True), (700, 2048, True), (64, 5120, True)])
def test_norm(m, k, res):
    x, r = rows16(k, m, k, 0.5), (rows16(k + 1, m, k, 2.0) if res else None)
    gamma = (1 + 0.2 * torch.randn(k, generator=gen(5))).half()
    eps = 1e-5
    h, c, s = q.residual_rmsnorm_mxfp8(x.cuda(), gamma.cuda(), None if r is None else r.cuda(), eps)
    want_h = x if r is None else (x.float() + r.float()).half()
    assert torch.equal(h.cpu(), want_h)
    f = want_h.double()
    n = f / torch.sqrt((f * f).mean(-1, keepdim=True) + eps) * gamma.double()
    # the mean's fp32 sum in at most 64 steps a thread and a tree, the root, the products:
    # 2^-20 of the value at most (half of the sum's relative error reaches the root)
    ref.check_mx8(c.cpu(), s.cpu(), n, 2.0 ** -18 * n.abs(), "norm")


def test_norm_in_place_and_not_finite():
    x, r, gamma = rows16(1, 6, 512), rows16(2, 6, 512), torch.ones(512).half()
    want = q.residual_rmsnorm_mxfp8(x.cuda(), gamma.cuda(), r.cuda())
    for at in (0, 1):
        xd, rd = x.cuda(), r.cuda()
        h, c, s = q.residual_rmsnorm_mxfp8(xd, gamma.cuda(), rd, h=(xd, rd)[at])
        assert h.data_ptr() == (xd, rd)[at].data_ptr()
        assert all(torch.equal(a, b) for a, b in zip((h, c, s), want))
    x[1, 3], x[2, 100] = float("nan"), float("inf")
    _, c, s = q.residual_rmsnorm_mxfp8(x.cuda(), gamma.cuda(), r.cuda())
    assert bool((s[1] == 255).all()) and int(s[2, 100 // 32]) == 255
    keep = [0, 3, 4, 5]
    assert torch.equal(c[keep], want[1][keep]) and torch.equal(s[keep], want[2][keep])
    z, c, s = q.residual_rmsnorm_mxfp8(torch.zeros(2, 64).half().cuda(), gamma[:64].cuda())
    assert int(s.max()) == 0 and bool((q.mx_dequantize(c, s) == 0).all())


# ----------------------------------------------------------------- products

SIZES = [(1, 32), (7, 64), (64, 96), (127, 128), (128, 160), (129, 256), (200, 1120), (1003, 512), (40, 4096), (256, 2080),
         (391, 1408), (512, 6016)]


@pytest.mark.parametrize("n,k", SIZES)
@pytest.mark.parametrize("m", [1, 2, 3, 5, 8])
def test_matvec(m, n, k):
    w, x = weight(n + k, n, k), rows16(m + k, m, k)
    y = q.qgemv_mxfp4(dev(w), x.cuda())
    want, tol = ref.product(w, x.double())
    # fp16 rows are held to 2^-26 of their block's largest value
    wide = x.double().unflatten(-1, (-1, 32)).abs().amax(-1).repeat_interleave(32, -1)
    tol = tol + 2.0 ** -26 * (wide @ ref.values(*w).abs().T)
    ref.near(y, want, tol, "matvec")
    r = rows16(n, m, n)
    rd = r.cuda()
    y2 = q.qgemv_mxfp4(dev(w), x.cuda(), residual=rd, y=rd)
    assert y2.data_ptr() == rd.data_ptr()
    ref.near(y2, want + r.double(), tol + 2.0 ** -23 * (want + r.double()).abs(), "matvec + residual")


@pytest.mark.parametrize("n,k", SIZES)
@pytest.mark.parametrize("m", [1, 8, 15, 17, 33, 100, 129, 260])
def test_product(m, n, k):
    w, x = weight(n + k, n, k), acts(m + k, m, k)
    y = q.mx_gemm(dev(w), dev(x))
    want, tol = ref.product(w, ref.values(*x))
    ref.near(y, want, tol, "product")
    r = rows16(n, m, n)
    rd = r.cuda()
    q.mx_gemm(dev(w), dev(x), residual=rd, y=rd)
    ref.near(rd, want + r.double(), tol + 2.0 ** -23 * (want + r.double()).abs(), "product + residual")
    assert q.device_status() == 0


@pytest.mark.parametrize("n,k", [(32, 32), (7, 64), (96, 96), (129, 128), (128, 160), (416, 1120), (992, 512), (160, 4096),
                                 (288, 1408)])
@pytest.mark.parametrize("m", [1, 8, 17, 50, 129, 200])
def test_gated(m, n, k):
    wg, wu, x = weight(n + k, n, k), weight(n + k + 1, n, k), acts(m + k, m, k)
    xv = ref.values(*x)
    want, tol = ref.gated(*ref.product(wg, xv), *ref.product(wu, xv))
    h = torch.zeros(m, n, dtype=torch.float16, device="cuda")
    q.mx_swiglu(dev(wg), dev(wu), dev(x), h=h)
    ref.near(h, want, tol, "gated")
    if n % 32 == 0:
        c, s = q.mx_swiglu(dev(wg), dev(wu), dev(x))
        ref.check_mx8(c.cpu(), s.cpu(), want, tol, "gated, MXFP8")
        h2 = torch.zeros_like(h)
        c2, s2 = q.mx_swiglu(dev(wg), dev(wu), dev(x), h=h2, codes=torch.zeros_like(c), scales=torch.zeros_like(s))
        assert torch.equal(c, c2) and torch.equal(s, s2) and torch.equal(h, h2)
    assert q.device_status() == 0


@pytest.mark.parametrize("m,n,k", [(1, 20000, 256), (3, 45000, 128), (20, 30000, 256), (1200, 1500, 256), (2100, 300, 160)])
def test_many_tiles(m, n, k):
    """More tiles than multiprocessors, several for a thread block."""
    w, x = weight(1, n, k), acts(2, m, k)
    y = q.mx_gemm(dev(w), dev(x))
    want, tol = ref.product(w, ref.values(*x))
    ref.near(y, want, tol, "product")
    if m <= 8:
        x16 = rows16(3, m, k)
        want, tol = ref.product(w, x16.double())
        ref.near(q.qgemv_mxfp4(dev(w), x16.cuda()), want, tol + 2.0 ** -20 * want.abs().max(), "matvec")


@pytest.mark.parametrize("m,n,k,gated", ref.PAIRS)
def test_pairs_of_blocks(m, n, k, gated):
    """Products that two thread blocks share, whose last tiles have rows and columns that there are not."""
    w, x = weight(m + n, n, k), acts(k, m, k)
    xv = ref.values(*x)
    want, tol = ref.product(w, xv)
    if gated:
        up = weight(m, n, k)
        want, tol = ref.gated(want, tol, *ref.product(up, xv))
        h = torch.zeros(m, n, dtype=torch.float16, device="cuda")
        q.mx_swiglu(dev(w), dev(up), dev(x), h=h)
        ref.near(h, want, tol, "gated")
        if n % 32 == 0:
            c, s = q.mx_swiglu(dev(w), dev(up), dev(x))
            ref.check_mx8(c.cpu(), s.cpu(), want, tol, "gated, MXFP8")
            h2, c2, s2 = torch.zeros_like(h), torch.zeros_like(c), torch.zeros_like(s)
            q.mx_swiglu(dev(w), dev(up), dev(x), h=h2, codes=c2, scales=s2)
            assert torch.equal(c, c2) and torch.equal(s, s2) and torch.equal(h, h2)
    else:
        y = q.mx_gemm(dev(w), dev(x))
        ref.near(y, want, tol, "product")
        r = rows16(n, m, n)
        rd = r.cuda()
        got = q.mx_gemm(dev(w), dev(x), residual=rd, y=rd)              # in place
        ref.near(got, want + r.double(), tol + 2.0 ** -23 * (want + r.double()).abs(), "product and residual")
        out = placed(torch.zeros(m, n).half(), 2)                       # (not written four at a time)
        assert torch.equal(q.mx_gemm(dev(w), dev(x), y=out), y)
        # scales that are not 4-byte aligned, and codes that are not 32-byte: blocks by themselves
        wd, xd = (placed(w[0], 16), placed(w[1], 1)), (x[0].cuda(), placed(x[1], 3))
        ref.near(q.mx_gemm(wd, xd), want, tol, "product of other alignments")
    assert q.device_status() == 0


@pytest.mark.parametrize("m,n,k,gated", ref.PAIRS_SMALL)
def test_pairs_write_nothing_else(m, n, k, gated):
    w, x = dev(weight(1, n, k)), dev(acts(2, m, k))

    def banded(shape, dtype):
        raw = torch.full((torch.Size(shape).numel() * torch.empty(0, dtype=dtype).element_size() + 4096,), 0xA5,
                         dtype=torch.uint8, device="cuda")
        return raw, raw[2048:-2048].view(dtype).view(shape)

    bands = [banded((m, n), torch.float16)]
    if gated and n % 32 == 0:
        bands += [banded((m, n), torch.uint8), banded((m, n // 32), torch.uint8)]
    kept = [t.clone() for t in (*w, *x)]
    if gated:
        q.mx_swiglu(w, w, x, h=bands[0][1], **({} if n % 32 else dict(codes=bands[1][1], scales=bands[2][1])))
    else:
        q.mx_gemm(w, x, y=bands[0][1])
        q.mx_gemm(w, x, residual=bands[0][1], y=bands[0][1])
    for raw, _ in bands:
        assert bool((raw[:2048] == 0xA5).all()) and bool((raw[-2048:] == 0xA5).all())
    assert all(torch.equal(a, b) for a, b in zip(kept, (*w, *x)))


def test_pairs_beyond_32_bits():
    """Outputs of more than 2^31 elements: the last rows against 64 bits."""
    g = torch.Generator(device="cuda").manual_seed(3)
    m, n, k = ref.PAIRS_LARGEST
    some = 70
    w, u = (q.mx_quantize(torch.randn(n, k, generator=g, device="cuda").half(), 4) for _ in range(2))
    x = q.mx_quantize(torch.randn(m, k, generator=g, device="cuda").half())
    tail = (x[0][-some:].cpu(), x[1][-some:].cpu())
    host = [(t[0].cpu(), t[1].cpu()) for t in (w, u)]
    want, tol = ref.product(host[0], ref.values(*tail))
    y = q.mx_gemm(w, x)
    assert y.numel() > 1 << 31
    ref.near(y[-some:], want, tol, "product")
    first = y[-some:].clone()
    q.mx_gemm(w, x, residual=y, y=y)
    both = want + first.cpu().double()
    ref.near(y[-some:], both, tol + 2.0 ** -23 * both.abs(), "product and residual")
    del y
    want, tol = ref.gated(want, tol, *ref.product(host[1], ref.values(*tail)))
    h = torch.empty(m, n, dtype=torch.float16, device="cuda")
    ref.near(q.mx_swiglu(w, u, x, h=h)[-some:], want, tol, "gated")
    del h
    n32 = n // 32 * 32
    c, s = q.mx_swiglu(*((t[0][:n32].contiguous(), t[1][:n32].contiguous()) for t in (w, u)), x)
    assert c.numel() > 1 << 31
    ref.check_mx8(c[-some:].cpu(), s[-some:].cpu(), want[:, :n32], tol[:, :n32], "gated, MXFP8")
    assert q.device_status() == 0
    del c, s
    torch.cuda.empty_cache()


def test_pairs_captured_and_replayed():
    """Of new values in the same tensors, and two of them on two streams at once."""
    m, n, k = ref.PAIRS_GRAPH
    w, u = dev(weight(1, n, k)), dev(weight(2, n, k))
    x = dev(acts(3, m, k))
    y, held = torch.zeros(m, n, dtype=torch.float16, device="cuda"), q.mx_swiglu(w, u, x)
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        q.mx_gemm(w, x, y=y)
        with torch.cuda.stream(side):
            q.mx_swiglu(w, u, x, codes=held[0], scales=held[1])
        torch.cuda.current_stream().wait_stream(side)
    for seed in (7, 8):
        for to, t in zip(x, acts(seed, m, k)):
            to.copy_(t)
        graph.replay()
        torch.cuda.synchronize()
        c, s = q.mx_swiglu(w, u, x)
        assert torch.equal(y, q.mx_gemm(w, x)) and torch.equal(held[0], c) and torch.equal(held[1], s)
    assert q.device_status() == 0


def test_products_of_every_code_and_scale():
    """Each weight code times each activation code, at scales from one end to the other."""
    k = 32
    wn = torch.zeros(16, k, dtype=torch.long)
    wn[:, 5] = torch.arange(16)
    x = torch.zeros(256, k, dtype=torch.uint8)
    x[:, 5] = torch.arange(256).to(torch.uint8)
    x = x[~torch.isnan(ref.E4M3[x[:, 5].long()])]
    for ws, xs in ((127, 127), (100, 150), (150, 104), (1, 250), (250, 1), (126, 128), (0, 252), (252, 0)):
        w = (ref.pack4(wn), torch.full((16, 1), ws, dtype=torch.uint8))
        xx = (x, torch.full((x.shape[0], 1), xs, dtype=torch.uint8))
        y = q.mx_gemm(dev(w), dev(xx))
        ref.near(y, ref.values(*xx) @ ref.values(*w).T, 0.0, f"scales {ws}, {xs}")


def test_fp16_rows_keep_their_bits():
    """One weight of 1 in each row: the product is the fp16 value itself, subnormals and
    the largest ones among them, to 2^-26 of the block's largest."""
    k = 64
    wn = torch.zeros(k, k, dtype=torch.long)
    wn[torch.arange(k), torch.arange(k)] = 2
    w = (ref.pack4(wn), torch.full((k, 2), 127, dtype=torch.uint8))
    g = gen(11)
    for scale in (1.0, 2.0 ** -14, 2.0 ** -22, 6.0e3):
        x = (torch.randn(8, k, generator=g) * scale).half()
        x[:, 0] = x[:, 32] = 0
        y = q.qgemv_mxfp4(dev(w), x.cuda()).cpu().double()
        wide = x.double().unflatten(-1, (-1, 32)).abs().amax(-1).repeat_interleave(32, -1)
        # (a difference below half a step of fp16 does not show)
        assert bool(((y - x.double()).abs() <= 2.0 ** -26 * wide).all())


def test_not_finite():
    n, k = 40, 256
    w, x = weight(1, n, k), acts(2, 12, k)
    base = q.mx_gemm(dev(w), dev(x)).cpu()
    w[1][7, 3] = 255
    x[1][4, 2] = 255
    x[0][5, 9] = 0x7F
    y = q.mx_gemm(dev(w), dev(x)).cpu()
    bad = torch.zeros(12, n, dtype=torch.bool)
    bad[4] = bad[5] = True
    bad[:, 7] = True
    assert torch.equal(torch.isnan(y), bad) and torch.equal(y[~bad], base[~bad])
    w = weight(1, n, k)
    x16 = rows16(3, 4, k)
    base = q.qgemv_mxfp4(dev(w), x16.cuda()).cpu()
    x16[1, 200], x16[2, 0] = float("inf"), float("nan")
    y = q.qgemv_mxfp4(dev(w), x16.cuda()).cpu()
    assert bool(torch.isnan(y[1:3]).all()) and torch.equal(y[[0, 3]], base[[0, 3]])


@pytest.mark.parametrize("k", [128, 512, 1120, 2048])
@pytest.mark.parametrize("offset", [16, 48, 128])
def test_alignments(k, offset):
    m, n = 21, 150
    w, x = weight(4, n, k), acts(5, m, k)
    want = q.mx_gemm(dev(w), dev(x))
    wd = (placed(w[0], offset), placed(w[1], offset // 16))
    xd = (placed(x[0], offset), placed(x[1], offset // 16 + 1))
    out = placed(torch.zeros(m, n).half(), 2)
    assert torch.equal(q.mx_gemm(wd, xd, y=out), want)
    x16 = rows16(6, 3, k)
    assert torch.equal(q.qgemv_mxfp4(wd, placed(x16, offset), y=placed(torch.zeros(3, n).half(), 6)),
                       q.qgemv_mxfp4(dev(w), x16.cuda()))
    # gate and up as the halves of one matrix
    both = (torch.cat([w[0], weight(8, n, k)[0]]).cuda(), torch.cat([w[1], weight(8, n, k)[1]]).cuda())
    got = q.mx_swiglu((both[0][:n], both[1][:n]), (both[0][n:], both[1][n:]), dev(x),
                      h=torch.zeros(m, n, dtype=torch.float16, device="cuda"))
    assert torch.equal(got, q.mx_swiglu(dev(w), dev(weight(8, n, k)), dev(x),
                                        h=torch.zeros(m, n, dtype=torch.float16, device="cuda")))


def test_nothing_else_is_written():
    m, n, k = 19, 96, 160
    w, x = dev(weight(1, n, k)), dev(acts(2, m, k))

    def banded(shape, dtype):
        raw = torch.full((torch.Size(shape).numel() * torch.empty(0, dtype=dtype).element_size() + 512,), 0xA5,
                         dtype=torch.uint8, device="cuda")
        return raw, raw[256:-256].view(dtype).view(shape)

    bands = {name: banded(s, t) for name, s, t in (
        ("y", (m, n), torch.float16), ("c", (m, n), torch.uint8), ("s", (m, n // 32), torch.uint8),
        ("h", (m, k), torch.float16), ("nc", (m, k), torch.uint8), ("ns", (m, k // 32), torch.uint8),
        ("qc", (m, k // 8), torch.int32), ("qs", (m, k // 32), torch.uint8), ("v", (m, k), torch.float16),
        ("z", (5, n), torch.float16))}
    kept = [t.clone() for t in (*w, *x)]
    x16, r16, gamma = rows16(3, m, k).cuda(), rows16(4, m, k).cuda(), torch.ones(k, device="cuda").half()
    q.mx_gemm(w, x, y=bands["y"][1])
    q.mx_swiglu(w, w, x, codes=bands["c"][1], scales=bands["s"][1])
    q.residual_rmsnorm_mxfp8(x16, gamma, r16, h=bands["h"][1], codes=bands["nc"][1], scales=bands["ns"][1])
    q.mx_quantize(x16, 4, codes=bands["qc"][1], scales=bands["qs"][1])
    q.mx_dequantize(bands["qc"][1], bands["qs"][1], out=bands["v"][1])
    q.qgemv_mxfp4(w, x16[:5], y=bands["z"][1])
    for name, (raw, _) in bands.items():
        assert bool((raw[:256] == 0xA5).all()) and bool((raw[-256:] == 0xA5).all()), name
    assert all(torch.equal(a, b) for a, b in zip(kept, (*w, *x)))


# ---------------------------------------------------------- as they are used

def layer(seed, hidden, inter):
    g = gen(seed)
    make = lambda n, k: q.mx_quantize((torch.randn(n, k, generator=g) * k ** -0.5).half().cuda(), 4)  # noqa: E731
    return dict(gate=make(inter, hidden), up=make(inter, hidden), down=make(hidden, inter),
                gamma=(1 + 0.1 * torch.randn(hidden, generator=g)).half().cuda())


def block(L, x, r, out=None):
    """A pre-norm gated block: what a layer does behind its attention."""
    h, c, s = q.residual_rmsnorm_mxfp8(x, L["gamma"], r)
    return q.mx_gemm(L["down"], q.mx_swiglu(L["gate"], L["up"], (c, s)), residual=h, y=out)


@pytest.mark.parametrize("m", [1, 8, 40, 300])
def test_gated_block(m):
    hidden, inter = 512, 1440
    L = layer(1, hidden, inter)
    x, r = rows16(2, m, hidden, 0.5).cuda(), rows16(3, m, hidden, 0.5).cuda()
    got = block(L, x, r)
    # each step against its form in 64 bits, fed with what the step before gave
    h, c, s = q.residual_rmsnorm_mxfp8(x, L["gamma"], r)
    hc, hs = q.mx_swiglu(L["gate"], L["up"], (c, s))
    cpu = lambda p: tuple(t.cpu() for t in p)  # noqa: E731
    xv = ref.values(c.cpu(), s.cpu())
    want, tol = ref.gated(*ref.product(cpu(L["gate"]), xv), *ref.product(cpu(L["up"]), xv))
    ref.check_mx8(hc.cpu(), hs.cpu(), want, tol, "gated")
    want, tol = ref.product(cpu(L["down"]), ref.values(hc.cpu(), hs.cpu()))
    ref.near(got, want + h.cpu().double(), tol + 2.0 ** -23 * (want + h.cpu().double()).abs(), "block")
    assert torch.equal(got, block(L, x, r))                     # the same bits every time


def test_decode_and_batch_agree():
    """fp16 rows and the same rows in MXFP8, where those hold them exactly."""
    n, k = 300, 1024
    w = dev(weight(1, n, k))
    x = q.mx_dequantize(*q.mx_quantize(rows16(2, 8, k).cuda(), 8))
    a, b = q.qgemv_mxfp4(w, x), q.mx_gemm(w, q.mx_quantize(x, 8))
    want, tol = ref.product(tuple(t.cpu() for t in w), x.cpu().double())
    ref.near(a, want, tol, "decode")
    ref.near(b, want, tol, "batch")
    assert torch.equal(q.qgemv_mxfp4(w, x[3]), a[3])            # a row does not depend on the others


def test_captured_and_replayed():
    L = layer(4, 384, 1024)
    m = 24
    x, r = rows16(5, m, 384).cuda(), rows16(6, m, 384).cuda()
    out = torch.zeros(m, 384, dtype=torch.float16, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        block(L, x, r, out)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        block(L, x, r, out)
        first = q.qgemv_mxfp4(L["down"], q.mx_dequantize(*q.mx_swiglu(L["gate"], L["up"], q.mx_quantize(x[:4]))))
    for seed in (7, 8):
        x.copy_(rows16(seed, m, 384))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, block(L, x, r))
        assert torch.equal(first, q.qgemv_mxfp4(L["down"], q.mx_dequantize(
            *q.mx_swiglu(L["gate"], L["up"], q.mx_quantize(x[:4])))))


def test_streams_and_fresh_weights():
    """Two streams at once, each with weights quantised right before the product."""
    g = gen(9)
    k, n, m = 1024, 640, 70
    raw = [(torch.randn(n, k, generator=g) * k ** -0.5).half().cuda() for _ in range(2)]
    x = dev(acts(10, m, k))
    x16 = rows16(11, 3, k).cuda()
    want = [(q.mx_gemm(q.mx_quantize(w, 4), x), q.qgemv_mxfp4(q.mx_quantize(w, 4), x16)) for w in raw]
    streams = [torch.cuda.Stream() for _ in range(2)]
    held = [(torch.zeros(n, k // 8, dtype=torch.int32, device="cuda"), torch.zeros(n, k // 32, dtype=torch.uint8, device="cuda"))
            for _ in range(2)]
    torch.cuda.synchronize()
    got = [None, None]
    for _ in range(20):
        for i, st in enumerate(streams):
            held[i][0].record_stream(st)
            with torch.cuda.stream(st):
                held[i][0].zero_()
            w = q.mx_quantize(raw[i], 4, codes=held[i][0], scales=held[i][1], stream=st)
            got[i] = (q.mx_gemm(w, x, stream=st), q.qgemv_mxfp4(w, x16, stream=st))
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert all(torch.equal(u, v) for u, v in zip(a, b))
    assert q.device_status() == 0


def test_shapes_and_no_rows():
    w = dev(weight(1, 96, 64))
    x = torch.zeros(0, 64, dtype=torch.float16, device="cuda")
    c, s = q.mx_quantize(x)
    assert c.shape == (0, 64) and s.shape == (0, 2)
    assert q.mx_dequantize(c, s).shape == (0, 64)
    assert q.mx_gemm(w, (c, s)).shape == (0, 96)
    assert q.mx_swiglu(w, w, (c, s))[0].shape == (0, 96)
    assert q.residual_rmsnorm_mxfp8(x, torch.ones(64, device="cuda").half())[1].shape == (0, 64)
    x = rows16(1, 6, 64).cuda()
    c, s = q.mx_quantize(x.view(2, 3, 64))
    assert c.shape == (2, 3, 64) and s.shape == (2, 3, 2)
    assert torch.equal(q.mx_gemm(w, (c, s)).view(6, 96), q.mx_gemm(w, q.mx_quantize(x)))
    assert torch.equal(q.mx_gemm(w, (c.view(torch.float8_e4m3fn), s)).view(6, 96), q.mx_gemm(w, q.mx_quantize(x)))
    assert q.qgemv_mxfp4(w, x[0]).shape == (96,) and q.mx_gemm(w, (c[0, 0], s[0, 0])).shape == (96,)


def test_refusals():
    w = dev(weight(1, 96, 64))
    x = rows16(1, 9, 64).cuda()
    xq = q.mx_quantize(x)
    for call in (lambda: q.qgemv_mxfp4(w, x),                          # nine rows
                 lambda: q.mx_quantize(x[:, :48].contiguous()),        # half a block
                 lambda: q.mx_swiglu((w[0][:90], w[1][:90]), (w[0][:90], w[1][:90]), xq)):
        with pytest.raises(q.QgemvError):
            call()
    for call in (lambda: q.mx_quantize(x, 5), lambda: q.mx_quantize(x.t()), lambda: q.mx_quantize(x.cpu()),
                 lambda: q.mx_gemm(w, (xq[0][:, :32].contiguous(), xq[1])), lambda: q.mx_gemm(w, (xq[0], xq[1][:4])),
                 lambda: q.mx_gemm((w[0], w[1][:5]), xq), lambda: q.mx_gemm(w, xq, y=torch.zeros(9, 95, device="cuda").half()),
                 lambda: q.mx_gemm(w, xq, residual=torch.zeros(8, 96, device="cuda").half()),
                 lambda: q.qgemv_mxfp4(w, x[:2, :32].contiguous()), lambda: q.mx_dequantize(xq[0], xq[1][:, :1]),
                 lambda: q.residual_rmsnorm_mxfp8(x, torch.ones(32, device="cuda").half()),
                 lambda: q.mx_swiglu(w, (w[0][:64], w[1][:64]), xq)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: q.mx_quantize(x.float()), lambda: q.mx_gemm(w, (xq[0].int(), xq[1])),
                 lambda: q.qgemv_mxfp4((w[0], w[1].int()), x[:2])):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(q.QgemvError):
        q.residual_rmsnorm_mxfp8(x, torch.ones(64, device="cuda").half(), eps=0.0)


# -------------------------------------------------------- the largest, and any

def test_longest_fp16_rows():
    k = 28672
    w, x = weight(1, 33, k), rows16(2, 8, k, 0.05)
    y = q.qgemv_mxfp4(dev(w), x.cuda())
    want, tol = ref.product(w, x.double())
    wide = x.double().unflatten(-1, (-1, 32)).abs().amax(-1).repeat_interleave(32, -1)
    ref.near(y, want, tol + 2.0 ** -26 * (wide @ ref.values(*w).abs().T), "matvec")
    assert torch.equal(q.qgemv_mxfp4(dev(w), x[2:4].cuda()), y[2:4])
    with pytest.raises(q.QgemvError):
        q.qgemv_mxfp4(dev(weight(1, 4, k + 32)), torch.zeros(1, k + 32, dtype=torch.float16, device="cuda"))


def test_long_rows():
    k = 70016                                                    # 547 steps, no whole groups of four
    w, x = weight(3, 20, k), acts(4, 3, k)
    want, tol = ref.product(w, ref.values(*x))
    ref.near(q.mx_gemm(dev(w), dev(x)), want, tol, "product")
    want, tol = ref.gated(want, tol, want, tol)
    h = torch.zeros(3, 20, dtype=torch.float16, device="cuda")
    ref.near(q.mx_swiglu(dev(w), dev(w), dev(x), h=h), want, tol, "gated")


def test_offsets_beyond_32_bits():
    """More than 2^32 values quantised, outputs and weights of more than 2^31 elements: the
    last rows against the same rows alone."""
    g = torch.Generator(device="cuda").manual_seed(1)
    m, k = 140000, 32768
    x = torch.empty(m, k, dtype=torch.float16, device="cuda")
    x[-300:] = torch.randn(300, k, generator=g, device="cuda").half()
    x[:-300] = 1.0
    for bits in (4, 8):
        c, s = q.mx_quantize(x, bits)
        c2, s2 = q.mx_quantize(x[-300:].contiguous(), bits)
        assert torch.equal(c[-300:], c2) and torch.equal(s[-300:], s2) and int((s[:-300] != s[0, 0]).sum()) == 0
        v = q.mx_dequantize(c, s)
        assert torch.equal(v[-300:], q.mx_dequantize(c2, s2))
        del v
    h, nc, ns = q.residual_rmsnorm_mxfp8(x, torch.ones(k, device="cuda").half(), x)
    _, nc2, ns2 = q.residual_rmsnorm_mxfp8(x[-300:].contiguous(), torch.ones(k, device="cuda").half(), x[-300:].contiguous())
    assert torch.equal(nc[-300:], nc2) and torch.equal(ns[-300:], ns2)
    del h, nc, ns, x
    # weights of 2^32 codes, one row of x
    w = (c[:, :4096], s) if bits == 4 else q.mx_quantize(torch.randn(300, k, generator=g, device="cuda").half(), 4)
    big = (w[0].repeat(470, 1), w[1].repeat(470, 1))
    xs = q.mx_quantize(torch.randn(2, k, generator=g, device="cuda").half())
    y, y2 = q.mx_gemm(big, xs), q.mx_gemm(w, xs)
    assert big[0].numel() * 8 > 1 << 32
    near = (y[:, -300:].float() - y2.float()).abs().max() <= 2e-3 * y2.float().abs().max()
    assert bool(near) and torch.equal(y[:, :300], y[:, 300:600])
    del big, y
    # outputs of 2^31 elements and more
    n, m, k = 50000, 45000, 32
    w = q.mx_quantize(torch.randn(n, k, generator=g, device="cuda").half(), 4)
    xs = q.mx_quantize(torch.randn(m, k, generator=g, device="cuda").half())
    y = q.mx_gemm(w, xs)
    last = q.mx_gemm(w, (xs[0][-50:].contiguous(), xs[1][-50:].contiguous()))
    assert y.numel() > 1 << 31 and torch.equal(y[-50:], last)
    q.mx_gemm(w, xs, residual=y, y=y)
    assert torch.equal(y[-50:], q.mx_gemm(w, (xs[0][-50:].contiguous(), xs[1][-50:].contiguous()), residual=last))
    del y
    nn = n // 32 * 32
    w = (w[0][:nn].contiguous(), w[1][:nn].contiguous())
    c, s = q.mx_swiglu(w, w, xs)
    c2, s2 = q.mx_swiglu(w, w, (xs[0][-50:].contiguous(), xs[1][-50:].contiguous()))
    assert torch.equal(c[-50:], c2) and torch.equal(s[-50:], s2)
    assert q.device_status() == 0
    torch.cuda.empty_cache()


@pytest.mark.parametrize("seed", range(30))
def test_any_size(seed):
    import random
    r = random.Random(seed)
    n, k = int(2 ** r.uniform(0, 10.5)), 32 * int(2 ** r.uniform(0, 7))
    m = int(2 ** r.uniform(0, 9.5))
    w, x = weight(seed, n, k), acts(seed, m, k)
    res = rows16(seed, m, n) if r.random() < 0.5 else None
    want, tol = ref.product(w, ref.values(*x))
    y = q.mx_gemm(dev(w), dev(x), residual=None if res is None else res.cuda())
    extra = 0 if res is None else res.double()
    ref.near(y, want + extra, tol + 2.0 ** -23 * (want + extra).abs(), "product")
    u = weight(seed + 100, n, k)
    want, tol = ref.gated(want, tol, *ref.product(u, ref.values(*x)))
    if n % 32 == 0:
        c, s = q.mx_swiglu(dev(w), dev(u), dev(x))
        ref.check_mx8(c.cpu(), s.cpu(), want, tol, "gated")
    else:
        ref.near(q.mx_swiglu(dev(w), dev(u), dev(x), h=torch.zeros(m, n, dtype=torch.float16, device="cuda")), want, tol, "gated")
    x16 = rows16(seed, min(m, 8), k)
    want, tol = ref.product(w, x16.double())
    wide = x16.double().unflatten(-1, (-1, 32)).abs().amax(-1).repeat_interleave(32, -1)
    ref.near(q.qgemv_mxfp4(dev(w), x16.cuda()), want, tol + 2.0 ** -26 * (wide @ ref.values(*w).abs().T), "matvec")


def test_cluster_and_ring_sizes():
    """Few tiles and long rows: the ways K is shared, with rows of x from one to a tile's."""
    for m, n, k in ((1, 96, 8192), (8, 224, 16384), (16, 128, 14336), (40, 160, 9216), (64, 128, 4096)):
        w, u, x = weight(m, n, k, 1), weight(m + 1, n, k, 1), acts(m, m, k)
        x = (x[0], (x[1].int() - 4).clamp(min=0).to(torch.uint8))
        xv = ref.values(*x)
        g, tg = ref.product(w, xv)
        ref.near(q.mx_gemm(dev(w), dev(x)), g, tg, f"product {m} {n} {k}")
        want, tol = ref.gated(g, tg, *ref.product(u, xv))
        c, s = q.mx_swiglu(dev(w), dev(u), dev(x))
        ref.check_mx8(c.cpu(), s.cpu(), want, tol, f"gated {m} {n} {k}")
    assert q.device_status() == 0
