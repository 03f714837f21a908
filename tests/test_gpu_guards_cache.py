"""Guard bands around everything that the paged-cache operators write: outputs, the
workspace (of exactly the size that is asked for) and the pools lie between margins of a
byte pattern that has to be there afterwards, inputs have to be as they were, and the
outputs are checked against the 64-bit forms as elsewhere."""
import numpy as np
import pytest
import torch

import kv_reference as ref
from test_gpu_kv_cache import close, queries

pytestmark = pytest.mark.gpu

q = pytest.importorskip("bit_group_quantized_qgemv_gb300")

MARGIN, BYTE = 8192, 0xA5


class Bands:
    """Tensors between margins; check() looks at the margins and at what must not change."""

    def __init__(self):
        self.outs, self.ins = [], []

    def out(self, shape, dtype, fill=None):
        n = int(np.prod(shape)) * torch.empty(0, dtype=dtype).element_size()
        buf = torch.full((n + 2 * MARGIN,), BYTE, dtype=torch.uint8, device="cuda")
        t = buf[MARGIN:MARGIN + n].view(dtype).view(shape)
        if fill is not None:
            t.copy_(fill)
        self.outs.append((buf, n))
        return t

    def given(self, t):
        d = t.cuda()
        self.ins.append((d, d.clone()))
        return d

    def check(self):
        torch.cuda.synchronize()
        for buf, n in self.outs:
            assert bool((buf[:MARGIN] == BYTE).all()) and bool((buf[MARGIN + n:] == BYTE).all())
        for d, was in self.ins:
            assert torch.equal(d.view(-1).view(torch.uint8), was.view(-1).view(torch.uint8))
        assert q.device_status() == 0


def cache_between(b, c):
    """The cache with its pools between margins."""
    k, v = (b.out(t.shape, torch.float16, t) for t in (c.k, c.v))
    return q.kv_cache(k, v, b.given(c.table), b.given(c.lens))


ATTENTION = [
    # hd, page, n_q, n_kv, sequences, page-table columns that no sequence needs
    (64, 16, 6, 2, [(1, 3000), (2, 700), (0, 50), (1, 1)], 1000),   # runs and a join over the units
    (128, 16, 48, 16, [(1, 100 + 13 * i) for i in range(40)], 0),   # more units than blocks
    (128, 32, 8, 1, [(4, 2000), (3, 15000)], 0),                    # 32 rows
    (64, 16, 5, 1, [(5, 1300), (3, 14001)], 0),                     # 25 rows
    (128, 16, 6, 2, [(1, 500)], 0),                                 # a cluster
    (128, 64, 7, 1, [(40, 9000), (3, 17)], 1),                      # many rows in parts, groups of 7
    (64, 16, 3, 1, [(211, 6000)], 1),                               # groups of 3
    (64, 16, 10, 2, [(130, 260), (1, 9), (77, 77)], 1),             # whole units, groups of 5
    (128, 256, 6, 1, [(50, 50), (129, 300)], 0),
]


@pytest.mark.parametrize("case", range(len(ATTENTION)))
def test_attention_and_mass_write_only_their_outputs(case):
    hd, page, n_q, n_kv, seqs, extra = ATTENTION[case]
    c = ref.make_cache(100 + case, seqs, n_kv, hd, page, extra_pages=extra)
    T, max_q, scale = sum(m for m, _ in seqs), max(m for m, _ in seqs), hd ** -0.5
    x = queries(100 + case, T, n_q, hd)
    b = Bands()
    h, xd, qs = cache_between(b, c), b.given(x), b.given(c.q_start)
    pools = h.k.clone(), h.v.clone()
    want, want_lse, tol, lse_tol = ref.attention(c, x, scale)
    n = q.paged_attention_workspace_bytes(h, T, n_q, max_q)
    for size in {n, 0}:
        out, lse = b.out((T, n_q, hd), torch.float16), b.out((T, n_q), torch.float32)
        err = b.out((1,), torch.int32, torch.zeros(1, dtype=torch.int32))
        ws = b.out((size,), torch.uint8)
        q.paged_attention(h, xd, qs, max_q=max_q, out=out, lse=lse, workspace=ws, err_flag=err)
        b.check()
        close(out, want, tol, "out")
        close(lse, want_lse, lse_tol, "lse")
        assert int(err) == 0
    mass = torch.rand(len(seqs), n_kv, c.cap, generator=torch.Generator().manual_seed(case))
    got = b.out(mass.shape, torch.float32, torch.full_like(mass, -7.0))
    ld = b.given(lse.cpu())
    q.attention_mass(h, xd, qs, ld, max_q=max_q, mass=b.given(mass), mass_out=got, err_flag=err)
    b.check()
    want_m, tol_m = ref.attention_mass(c, x, lse.cpu(), scale, mass)
    for s, (_, m) in enumerate(seqs):
        close(got[s, :, :m], want_m[s, :, :m], tol_m[s, :, :m], f"mass of sequence {s}")
        assert bool((got[s, :, m:] == -7.0).all())
    assert torch.equal(h.k.view(torch.int16), pools[0].view(torch.int16))
    assert torch.equal(h.v.view(torch.int16), pools[1].view(torch.int16))
    assert int(err) == 0


@pytest.mark.parametrize("hd,page,n_q,n_kv,rd,norm,seqs", [
    (128, 16, 5, 5, 128, True, [(1, 16)]),
    (64, 16, 9, 3, 24, False, [(3, 17), (0, 4), (30, 48)]),
    (128, 256, 7, 1, 0, True, [(200, 256), (1, 1)]),
    (64, 32, 32, 8, 64, True, [(1, 32)] * 61),
])
def test_rope_append_writes_only_the_new_entries(hd, page, n_q, n_kv, rd, norm, seqs):
    c = ref.make_cache(rd, seqs, n_kv, hd, page, spare=0, extra_pages=0)
    T, g = sum(m for m, _ in seqs), torch.Generator().manual_seed(rd)
    qkv = torch.randn(T, n_q + 2 * n_kv, hd, generator=g).half()
    pos = torch.randint(0, 5000, (T,), generator=g, dtype=torch.int32)
    inv = 1e4 ** (-torch.arange(0, rd, 2).float() / max(rd, 1))
    gamma = [torch.rand(hd, generator=g).half() if norm else None for _ in range(2)]
    b = Bands()
    h = cache_between(b, c)
    k, v = h.k.cpu(), h.v.cpu()
    out = b.out((T, n_q * hd), torch.float16)
    shape = (len(seqs), n_kv, c.cap)
    epos = b.out(shape, torch.int32, torch.full(shape, -9, dtype=torch.int32))
    emass = b.out(shape, torch.float32, torch.full(shape, 4.0))
    err = b.out((1,), torch.int32, torch.zeros(1, dtype=torch.int32))
    q.qk_norm_rope_append(h, b.given(qkv.view(T, -1)), b.given(c.q_start), b.given(pos),
                          b.given(inv) if rd else None, q_norm=b.given(gamma[0]) if norm else None,
                          k_norm=b.given(gamma[1]) if norm else None, q_out=out, entry_pos=epos,
                          entry_mass=emass, err_flag=err)
    b.check()
    new = torch.zeros(shape, dtype=torch.bool)
    for s, a, m, n in c.spans():
        for i in range(m):
            t, e = a + i, n - m + i
            want, tol = ref.rope(qkv[t, :n_q], int(pos[t]), inv.tolist(), gamma[0], 1e-6, False)
            close(out[t].view(n_q, hd), want, tol, f"query {t}")
            want, tol = ref.rope(qkv[t, n_q:n_q + n_kv], int(pos[t]), inv.tolist(), gamma[1], 1e-6, False)
            p, r = c.entry(s, e)
            close(h.k[p, :, r], want, tol, f"key {t}")
            k[p, :, r], v[p, :, r] = h.k[p, :, r].cpu(), qkv[t, n_q + n_kv:]
            new[s, :, e] = True
            assert bool((epos[s, :, e] == int(pos[t])).all())
    assert torch.equal(h.k.cpu().view(torch.int16), k.view(torch.int16))
    assert torch.equal(h.v.cpu().view(torch.int16), v.view(torch.int16))
    assert bool((epos.cpu()[~new] == -9).all()) and int(err) == 0
    assert torch.equal(emass.cpu(), torch.where(new, 0.0, 4.0))


@pytest.mark.parametrize("hd,page,n_kv,lens,keep,extra", [
    (64, 16, 2, [1000, 37, 0], 300, 0),             # the movers' list in shared memory
    (128, 16, 3, [160, 161], 160, 0),               # one mover
    (64, 16, 1, [128], 128, 0),                     # nothing to choose, a full table
    (64, 16, 8, [300 + 7 * i for i in range(24)], 200, 0),   # more heads than multiprocessors
    (64, 256, 2, [900, 30], 77, 310),               # keys made anew at every pass
    (128, 32, 1, [500], 1000, 0),                   # room for more than there is
])
def test_evict_writes_only_its_outputs(hd, page, n_kv, lens, keep, extra):
    c = ref.make_cache(keep, [(0, n) for n in lens], n_kv, hd, page, spare=0 if extra == 0 else 2,
                       extra_pages=extra)
    S, g = len(lens), torch.Generator().manual_seed(keep)
    mass = torch.floor(torch.rand(S, n_kv, c.cap, generator=g) * 50)
    pos = torch.argsort(torch.rand(S, n_kv, c.cap, generator=g), -1).int()
    nxt = torch.tensor([n + 3 for n in lens], dtype=torch.int32)
    b = Bands()
    h = cache_between(b, c)
    k, v = h.k.cpu(), h.v.cpu()
    kept = b.out((S, n_kv, keep), torch.int32)
    mo = b.out(mass.shape, torch.float32, torch.full_like(mass, -3.0))
    po = b.out(pos.shape, torch.int32, torch.full_like(pos, -3))
    left = b.out((S,), torch.int32)
    err = b.out((1,), torch.int32, torch.zeros(1, dtype=torch.int32))
    q.cache_evict(h, b.given(mass), b.given(pos), b.given(nxt), keep, n_sink=2, n_recent=5, kept=kept,
                  mass_out=mo, pos_out=po, kv_len_out=left, err_flag=err)
    b.check()
    want, want_left = ref.evict(c, mass, pos, nxt, keep, 2, 5)
    assert left.tolist() == want_left and int(err) == 0 and torch.equal(kept.cpu(), want)
    for s, n in enumerate(want_left):
        for hh in range(n_kv):
            src = want[s, hh, :n].long()
            assert torch.equal(mo[s, hh, :n].cpu(), mass[s, hh, src])
            assert torch.equal(po[s, hh, :n].cpu(), pos[s, hh, src])
            assert bool((mo[s, hh, n:] == -3.0).all()) and bool((po[s, hh, n:] == -3).all())
            for i in (src != torch.arange(n)).nonzero().view(-1).tolist():
                (pa, ra), (pb, rb) = c.entry(s, int(src[i])), c.entry(s, i)
                k[pb, hh, rb], v[pb, hh, rb] = c.k[pa, hh, ra], c.v[pa, hh, ra]
    assert torch.equal(h.k.cpu().view(torch.int16), k.view(torch.int16))
    assert torch.equal(h.v.cpu().view(torch.int16), v.view(torch.int16))
