"""Products with MXFP4 weights by clusters of blocks, and by blocks, with several tiles each, against plain 64-bit
forms, with guard bands around what they write."""
import pytest
import torch

import mx_reference as ref
from mx_cluster_shapes import ALONE, PAIRS_ODD, ROWS_ODD, SHARED

pytestmark = pytest.mark.gpu

q = pytest.importorskip("bit_group_quantized_qgemv_gb300")

BAND = 2048


def dev(pair):
    return tuple(t.cuda() for t in pair)


def weight(seed, n, k):
    g = torch.Generator().manual_seed(seed)
    return (ref.pack4(torch.randint(0, 16, (n, k), generator=g)),
            torch.randint(119, 125, (n, k // 32), generator=g).to(torch.uint8))


def rows16(seed, m, k):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(m, k, generator=g) * torch.exp(0.8 * torch.randn(k, generator=g))).half()


def acts(seed, m, k):
    c, s = ref.quantize(rows16(seed, m, k).double(), 8)
    return c.to(torch.uint8), s


class Banded:
    """A tensor on the GPU, `offset` bytes behind a 256-byte boundary, in memory with a known rest."""

    def __init__(self, shape, dtype, offset=0, like=None):
        size = torch.Size(shape).numel() * torch.empty(0, dtype=dtype).element_size()
        self.raw = torch.full((size + 2 * BAND + 256,), 0xA5, dtype=torch.uint8, device="cuda")
        self.at = BAND + offset
        self.t = self.raw[self.at:self.at + size].view(dtype).view(shape)
        if like is not None:
            self.t.copy_(like)

    def intact(self):
        end = self.at + self.t.numel() * self.t.element_size()
        return bool((self.raw[:self.at] == 0xA5).all()) and bool((self.raw[end:] == 0xA5).all())


@pytest.mark.parametrize("m,n,k,gated,fp16", [s for _, s in SHARED] + PAIRS_ODD + ALONE + ROWS_ODD)
def test_several_tiles_of_a_block(m, n, k, gated, fp16):
    w = weight(m + n, n, k)
    x = rows16(k, m, k) if fp16 else acts(k, m, k)
    want, tol = ref.product(w, x.double() if fp16 else ref.values(*x))
    wd, xd = dev(w), x.cuda() if fp16 else dev(x)
    if gated:
        up = weight(m, n, k)
        want, tol = ref.gated(want, tol, *ref.product(up, ref.values(*x)))
        ud = dev(up)
        h = Banded((m, n), torch.float16)
        q.mx_swiglu(wd, ud, xd, h=h.t)
        ref.near(h.t, want, tol, "gated")
        first = h.t.clone()
        q.mx_swiglu(wd, ud, xd, h=h.t)
        assert h.intact() and torch.equal(h.t, first)                    # the same bits every time
        if n % 32 == 0:
            c, s = Banded((m, n), torch.uint8), Banded((m, n // 32), torch.uint8, 3)
            q.mx_swiglu(wd, ud, xd, codes=c.t, scales=s.t)
            ref.check_mx8(c.t.cpu(), s.t.cpu(), want, tol, "gated, MXFP8")
            assert c.intact() and s.intact()
    else:
        call = q.qgemv_mxfp4 if fp16 else q.mx_gemm
        y = Banded((m, n), torch.float16)
        call(wd, xd, y=y.t)
        ref.near(y.t, want, tol, "product")
        first = y.t.clone()
        call(wd, xd, y=y.t)
        assert y.intact() and torch.equal(y.t, first)
        r = rows16(n, m, n)
        both = Banded((m, n), torch.float16, like=r)
        call(wd, xd, y=both.t, residual=both.t)                          # in place
        ref.near(both.t, want + r.double(), tol + 2.0 ** -23 * (want + r.double()).abs(), "product and residual")
        assert both.intact()
        # codes, scales and results of other alignments: other loads and stores, the same tiles
        wo = Banded(w[0].shape, torch.int32, 16, w[0]), Banded(w[1].shape, torch.uint8, 1, w[1])
        yo = Banded((m, n), torch.float16, 2)
        if fp16:
            call((wo[0].t, wo[1].t), xd, y=yo.t)
        else:
            xo = Banded(x[0].shape, torch.uint8, 16, x[0]), Banded(x[1].shape, torch.uint8, 3, x[1])
            call((wo[0].t, wo[1].t), (xo[0].t, xo[1].t), y=yo.t)
        ref.near(yo.t, want, tol, "product of other alignments")
        assert yo.intact()
    assert q.device_status() == 0


def test_two_streams_of_clusters():
    """Two products of several tiles a cluster at once, neither of which fits beside the other."""
    shapes = [SHARED[0][1], SHARED[5][1]]
    work = []
    for m, n, k, _, fp16 in shapes:
        w, x = dev(weight(m, n, k)), rows16(n, m, k).cuda() if fp16 else dev(acts(n, m, k))
        call = q.qgemv_mxfp4 if fp16 else q.mx_gemm
        work.append((call, w, x, call(w, x), [torch.empty(m, n, dtype=torch.float16, device="cuda") for _ in range(10)]))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in work]
    for i in range(10):
        for st, (call, w, x, _, outs) in zip(streams, work):
            call(w, x, y=outs[i], stream=st)
    torch.cuda.synchronize()
    for _, _, _, want, outs in work:
        assert all(torch.equal(o, want) for o in outs)
    assert q.device_status() == 0


@pytest.mark.parametrize("m,n,k", [s[:3] for s in ROWS_ODD])
def test_rows_of_an_odd_number_of_steps(m, n, k):
    """Many calls, each with rows of its own: those of the call before lie where these are taken apart to."""
    w = weight(n, n, k)
    wd, wv = dev(w), ref.values(*w).cuda()
    for seed in range(30):
        x = rows16(seed, m, k)
        xv = x.double().cuda()
        want = xv @ wv.T
        # (a step of 32 products is off by 2^-20 of the magnitudes so far at most: there are k / 32)
        tol = 2.0 ** -20 * (k // 32 + 1) * (xv.abs() @ wv.abs().T)
        ref.near(q.qgemv_mxfp4(wd, x.cuda()), want.cpu(), tol.cpu(), "product")
    assert q.device_status() == 0
