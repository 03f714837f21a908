"""The paged-cache operators (qk_norm_rope_append, paged_attention,
attention_mass, cache_evict) against plain 64-bit forms: lengths from zero,
odd sizes, head layouts, page sizes, rows and pages that must not matter
(filled with NaN and infinities), strides, bad pages, captured graphs, streams,
workspaces, and the four in a row as a decoding program uses them."""
import math

import numpy as np
import pytest
import torch

import kv_reference as ref
import synth
from qhelpers import dev_weight

pytestmark = pytest.mark.gpu

q = pytest.importorskip("bit_group_quantized_qgemv_gb300")


def handle(c):
    return q.kv_cache(c.k.cuda(), c.v.cuda(), c.table.cuda(), c.lens.cuda())


def queries(seed, T, n_q, hd, scale=2.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(T, n_q, hd, generator=g) * scale).half()


def close(got, want, tol, what):
    got = got.double().cpu()
    same = (got == want) | ((got - want).abs() <= tol)
    assert bool(same.all()), (f"{what}: {int((~same).sum())} of {same.numel()} outside, worst "
                              f"{float(((got - want).abs() / tol)[~same].max())} x tolerance")


ATTENTION = [
    # hd, page, n_q, n_kv, [(new tokens, length)]
    (128, 16, 4, 1, [(1, 1)]),
    (64, 16, 1, 1, [(1, 2), (0, 0), (1, 17)]),
    (128, 32, 8, 8, [(1, 15), (1, 16), (1, 31), (1, 33)]),
    (64, 64, 16, 2, [(1, 700), (1, 0), (1, 64), (0, 90)]),      # a token without entries
    (128, 16, 32, 8, [(1, 1111)]),
    (128, 64, 28, 4, [(1, 300), (2, 129)]),
    (128, 16, 12, 4, [(5, 77), (9, 9), (3, 400)]),              # 27 rows: two tiles of 16
    (64, 128, 10, 2, [(6, 513), (4, 4)]),
    (128, 256, 6, 2, [(4, 2), (7, 260)]),                       # more new tokens than entries
    (64, 16, 8, 2, [(33, 33), (8, 100)]),
    (128, 16, 8, 2, [(64, 200), (1, 65), (31, 31)]),
    (128, 64, 4, 4, [(130, 130), (127, 383)]),
    (64, 32, 14, 2, [(37, 300), (0, 10), (150, 150)]),
    (128, 32, 5, 1, [(61, 1000)]),
    (64, 256, 3, 3, [(257, 700)]),
]


@pytest.mark.parametrize("case", range(len(ATTENTION)))
def test_attention_and_mass(case):
    hd, page, n_q, n_kv, seqs = ATTENTION[case]
    c = ref.make_cache(case, seqs, n_kv, hd, page)
    T = sum(m for m, _ in seqs)
    x = queries(case, T, n_q, hd)
    scale = hd ** -0.5
    h = handle(c)
    xd, qs = x.cuda(), c.q_start.cuda()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    max_q = max(m for m, _ in seqs)
    out, lse = q.paged_attention(h, xd, qs, max_q=max_q, want_lse=True, err_flag=err)
    want, want_lse, tol, lse_tol = ref.attention(c, x, scale)
    close(out.view(T, n_q, hd), want, tol, "out")
    close(lse, want_lse, lse_tol, "lse")
    assert int(err) == 0
    # without a workspace, and with the default bound on the new tokens
    w0 = torch.empty(0, dtype=torch.uint8, device="cuda")
    out1, lse1 = q.paged_attention(h, xd.view(T, -1), qs, want_lse=True, workspace=w0)
    close(out1.view(T, n_q, hd), want, tol, "out, no workspace")
    close(lse1, want_lse, lse_tol, "lse, no workspace")

    g = torch.Generator().manual_seed(case)
    mass = torch.rand(len(seqs), n_kv, c.cap, generator=g)
    marked = torch.full_like(mass, -7.0).cuda()
    got = q.attention_mass(h, xd, qs, lse, max_q=max_q, mass=mass.cuda(), mass_out=marked, err_flag=err)
    want_m, tol_m = ref.attention_mass(c, x, lse.cpu(), scale, mass)
    for s, (_, n) in enumerate(seqs):
        close(got[s, :, :n], want_m[s, :, :n], tol_m[s, :, :n], f"mass of sequence {s}")
        assert bool((got[s, :, n:] == -7.0).all())
    # in place, and from nothing
    inplace = mass.cuda()
    q.attention_mass(h, xd, qs, lse, max_q=max_q, mass=inplace, mass_out=inplace)
    fresh = q.attention_mass(h, xd, qs, lse, max_q=max_q)
    for s, (_, n) in enumerate(seqs):
        assert torch.equal(inplace[s, :, :n], got[s, :, :n])
        assert torch.equal(inplace[s, :, n:], mass[s, :, n:].cuda())
        close(fresh[s, :, :n], want_m[s, :, :n] - mass[s, :, :n].double(), tol_m[s, :, :n], "mass from zero")
    assert int(err) == 0 and q.device_status() == 0


def _ragged(seed, n, most, longest):
    g = np.random.default_rng(seed)
    new = g.integers(0, most + 1, n)
    return [(int(m), int(m + g.integers(0, longest))) for m in new]


WIDE = [
    # hd, page, n_q, n_kv, sequences, page-table columns that no sequence needs
    (128, 16, 4, 2, [(1, 500)], 4000),                          # a table for 64,000 entries
    (64, 64, 6, 2, [(3, 700), (1, 90)], 3000),
    (128, 16, 8, 4, [(1, 6000), (2, 5000), (0, 7000), (1, 1)], 1),  # runs over the ends of units
    (64, 32, 24, 2, [(2, 9000)], 0),
    (64, 32, 24, 2, [(2, 13000)], 0),                           # 24 rows in many parts
    (128, 64, 8, 1, [(40, 9000)], 1),                           # 320 rows in many parts
    (64, 16, 4, 2, [(150, 3100), (20, 20)], 2000),
    (64, 16, 160, 1, [(1, 100), (2, 37)], 1),                   # 160 query heads to a key head
    (64, 16, 2, 1, _ragged(1, 40, 3, 200), 1),                  # more sequences than lanes
    (64, 16, 4, 2, _ragged(2, 40, 40, 300), 1),
    (128, 32, 4, 1, _ragged(3, 18, 60, 400), 20),
    (64, 16, 2, 2, [(0, 9)] * 70 + [(1, 33)] + [(0, 0)] * 40 + [(2, 5)], 1),
    (64, 16, 2, 2, [(0, 9)] * 70 + [(40, 333)] + [(0, 0)] * 40 + [(2, 5)], 1),
    (64, 16, 16, 16, _ragged(6, 24, 100, 300), 1),              # units for three rounds of blocks
    (64, 16, 8, 8, _ragged(7, 50, 60, 200), 1),
]


@pytest.mark.parametrize("case", range(len(WIDE)))
def test_wide_tables_many_sequences_and_many_parts(case):
    hd, page, n_q, n_kv, seqs, extra = WIDE[case]
    c = ref.make_cache(50 + case, seqs, n_kv, hd, page, extra_pages=extra)
    T, scale = sum(m for m, _ in seqs), hd ** -0.5
    x = queries(50 + case, T, n_q, hd)
    h, xd, qs = handle(c), x.cuda(), c.q_start.cuda()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    max_q = max(m for m, _ in seqs)
    want, want_lse, tol, lse_tol = ref.attention(c, x, scale)
    none = torch.empty(0, dtype=torch.uint8, device="cuda")
    for ws in (None, none):
        out, lse = q.paged_attention(h, xd, qs, max_q=max_q, want_lse=True, workspace=ws, err_flag=err)
        close(out.view(T, n_q, hd), want, tol, "out")
        close(lse, want_lse, lse_tol, "lse")
    got = q.attention_mass(h, xd, qs, lse, max_q=max_q, err_flag=err)
    want_m, tol_m = ref.attention_mass(c, x, lse.cpu(), scale, torch.zeros(len(seqs), n_kv, c.cap))
    close(got, want_m, tol_m, "mass")
    assert int(err) == 0 and q.device_status() == 0


def test_attention_weights_add_up():
    """Over the entries of a sequence the weights of its rows sum to one each."""
    hd, n_q, n_kv, seqs = 128, 8, 2, [(1, 5000), (40, 2100)]
    c = ref.make_cache(3, seqs, n_kv, hd, 16)
    x, qs, h = queries(3, 41, n_q, hd).cuda(), c.q_start.cuda(), handle(c)
    _, lse = q.paged_attention(h, x, qs, max_q=40, want_lse=True)
    m = q.attention_mass(h, x, qs, lse, max_q=40).double().sum(-1).cpu()
    rows = torch.tensor([[1.0], [40.0]]).double() * (n_q // n_kv)
    # lse and every weight each err by less than 1e-4 relative here (scores below 30)
    assert bool(((m - rows).abs() <= 2e-4 * rows).all())


def test_attention_strides_and_foreign_rows():
    """Rows before the first and behind the last sequence stay as they were;
    queries and outputs may lie in wider rows."""
    hd, n_q, n_kv = 64, 4, 2
    c = ref.make_cache(11, [(3, 40), (2, 7)], n_kv, hd, 16)
    c.q_start += 2
    T = 9
    wide = queries(11, T, n_q + 3, hd)
    x = wide[:, :n_q]
    xd = wide.cuda().view(T, -1)[:, :n_q * hd]
    buf = torch.full((T, n_q * hd + 24), 5.0, dtype=torch.float16, device="cuda")
    lse = torch.full((T, n_q), 9.0, device="cuda")
    q.paged_attention(handle(c), xd, c.q_start.cuda(), max_q=3, out=buf[:, :n_q * hd], lse=lse)
    want, want_lse, tol, lse_tol = ref.attention(c, x, hd ** -0.5)
    close(buf[2:7, :n_q * hd].reshape(5, n_q, hd), want[2:7], tol[2:7], "strided out")
    close(lse[2:7], want_lse[2:7], lse_tol[2:7], "lse")
    for rows in (slice(0, 2), slice(7, 9)):
        assert bool((buf[rows] == 5.0).all()) and bool((lse[rows] == 9.0).all())
    assert bool((buf[:, n_q * hd:] == 5.0).all())


@pytest.mark.parametrize("m,n", [(1, 90), (20, 90), (70, 90)])
@pytest.mark.parametrize("number", [-1, 1 << 20])
def test_bad_pages_are_masked(m, n, number):
    hd, n_q, n_kv = 128, 4, 2
    c = ref.make_cache(m, [(m, n), (m, n)], n_kv, hd, 16)
    c.table[0, 1] = number
    c.table[1, :] = number                       # this sequence sees nothing at all
    x = queries(m, 2 * m, n_q, hd)
    h, qs = handle(c), c.q_start.cuda()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = q.paged_attention(h, x.cuda(), qs, max_q=m, want_lse=True, err_flag=err)
    assert int(err) == 1
    want, want_lse, tol, lse_tol = ref.attention(c, x, hd ** -0.5)
    close(out.view(2 * m, n_q, hd), want, tol, "out")
    close(lse, want_lse, lse_tol, "lse")
    assert bool((out[m:] == 0).all()) and bool(torch.isneginf(lse[m:]).all())
    err.zero_()
    mass = torch.rand(2, n_kv, c.cap)
    got = q.attention_mass(h, x.cuda(), qs, lse, max_q=m, mass=mass.cuda(), err_flag=err)
    assert int(err) == 1
    want_m, tol_m = ref.attention_mass(c, x, lse.cpu(), hd ** -0.5, mass)
    close(got[:, :, :n], want_m[:, :, :n], tol_m[:, :, :n], "mass")


@pytest.mark.parametrize("m,n_q", [(6, 4), (40, 4), (200, 2)])
def test_hidden_infinities_do_not_leak(m, n_q):
    """An infinity or NaN in the key or value of one new token reaches that
    token and later ones, not the ones before it."""
    hd, n_kv, n = 128, 2, 230
    c = ref.make_cache(m, [(m, n)], n_kv, hd, 16)
    x = queries(m, m, n_q, hd)
    clean, _, tol, _ = ref.attention(c, x, hd ** -0.5)
    for what in ("k", "v"):
        d = ref.make_cache(m, [(m, n)], n_kv, hd, 16)
        pool = getattr(d, what)
        for back, value in ((m // 2, math.inf), (1, math.nan)):
            p, r = d.entry(0, n - back)
            pool[p, :, r, 3] = value
        out, _ = q.paged_attention(handle(d), x.cuda(), d.q_start.cuda(), max_q=m)
        before = m - m // 2                       # tokens that do not see the first of them
        close(out.view(m, n_q, hd)[:before], clean[:before], tol[:before], f"{what} hidden")
        if what == "v":
            assert not bool(torch.isfinite(out.view(m, n_q, hd)[m - 1, :, 3]).any())


def test_no_tokens_at_all():
    hd, n_q, n_kv = 64, 2, 1
    c = ref.make_cache(6, [(0, 20), (0, 3)], n_kv, hd, 16)
    h, qs = handle(c), c.q_start.cuda()
    none = torch.empty(0, n_q * hd, dtype=torch.float16, device="cuda")
    out, lse = q.paged_attention(h, none, qs, want_lse=True)
    assert out.shape == (0, n_q * hd) and lse.shape == (0, n_q)
    q.qk_norm_rope_append(h, torch.empty(0, 4 * hd, dtype=torch.float16, device="cuda"), qs,
                          torch.empty(0, dtype=torch.int32, device="cuda"))
    mass = torch.rand(2, n_kv, c.cap, device="cuda")
    got = q.attention_mass(h, none, qs, lse, mass=mass)
    assert torch.equal(got[0, :, :20], mass[0, :, :20]) and torch.equal(got[1, :, :3], mass[1, :, :3])


def test_more_new_tokens_than_declared():
    hd, n_q, n_kv = 64, 2, 1
    c = ref.make_cache(1, [(5, 20)], n_kv, hd, 16)
    x = queries(1, 5, n_q, hd)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full((5, n_q * hd), 3.0, dtype=torch.float16, device="cuda")
    q.paged_attention(handle(c), x.cuda(), c.q_start.cuda(), max_q=3, out=out, err_flag=err)
    want, _, tol, _ = ref.attention(c, x, hd ** -0.5)
    assert int(err) == 1
    close(out.view(5, n_q, hd)[:3], want[:3], tol[:3], "declared rows")
    assert bool((out[3:] == 3.0).all())


def test_lengths_and_starts_out_of_range_are_clamped():
    hd, n_q, n_kv, page = 64, 2, 2, 16
    c = ref.make_cache(2, [(1, 30), (1, 30)], n_kv, hd, page, extra_pages=0, poison=False)
    x = queries(2, 2, n_q, hd).cuda()
    h = handle(c)
    h.kv_len[:] = torch.tensor([1000, -5])        # capacity 32, nothing
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = q.paged_attention(h, x, c.q_start.cuda(), max_q=1, want_lse=True, err_flag=err)
    assert int(err) == 1 and bool((out[1] == 0).all()) and bool(torch.isneginf(lse[1]).all())
    c.lens = torch.tensor([32, 0], dtype=torch.int32)
    want, _, tol, _ = ref.attention(c, x.cpu(), hd ** -0.5)
    close(out.view(2, n_q, hd), want, tol, "clamped length")
    for starts in ([0, 5, 2], [-3, 1, 2], [0, 1, 1 << 30], [2, 1, 0]):
        err.zero_()
        q.paged_attention(h, x, torch.tensor(starts, dtype=torch.int32).cuda(), max_q=2, err_flag=err)
        q.attention_mass(h, x, torch.tensor(starts, dtype=torch.int32).cuda(), lse, max_q=2)
        assert int(err) == 1


ROPE = [
    # hd, page, n_q, n_kv, rotary, interleaved, norm, [(new, length)]
    (128, 16, 16, 8, 128, False, True, [(1, 1)]),
    (128, 16, 32, 8, 128, False, False, [(1, 17), (1, 16), (0, 3), (1, 400)]),
    (64, 32, 6, 2, 64, True, True, [(3, 35), (5, 5)]),
    (64, 16, 3, 3, 24, False, True, [(40, 41)]),
    (128, 64, 7, 1, 32, True, False, [(9, 70), (1, 1)]),
    (128, 128, 8, 4, 0, False, True, [(2, 2), (3, 300)]),
    (64, 256, 1, 1, 64, False, False, [(257, 300), (0, 0)]),
]


@pytest.mark.parametrize("case", range(len(ROPE)))
def test_rope_append(case):
    hd, page, n_q, n_kv, rd, inter, norm, seqs = ROPE[case]
    c = ref.make_cache(case, seqs, n_kv, hd, page)
    T = sum(m for m, _ in seqs)
    g = torch.Generator().manual_seed(case)
    qkv = (torch.randn(T, n_q + 2 * n_kv, hd, generator=g) * 1.5).half()
    pos = torch.randint(0, 1 << 20, (T,), generator=g, dtype=torch.int32)
    pos[0] = 0
    pos[-1] = 2 ** 31 - 1
    inv = (1e6 ** (-torch.arange(0, rd, 2).double() / max(rd, 1))).float()
    gq, gk = [(1 + 0.1 * torch.randn(hd, generator=g)).half() if norm else None for _ in range(2)]
    h = handle(c)
    before_k, before_v = h.k.clone(), h.v.clone()
    epos = torch.full((len(seqs), n_kv, c.cap), -9, dtype=torch.int32, device="cuda")
    emass = torch.full((len(seqs), n_kv, c.cap), 4.0, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    dev = lambda t: None if t is None else t.cuda()  # noqa: E731
    out = q.qk_norm_rope_append(h, qkv.view(T, -1).cuda(), c.q_start.cuda(), pos.cuda(),
                                inv.cuda() if rd else None, interleaved=inter, q_norm=dev(gq),
                                k_norm=dev(gk), eps=1e-6, entry_pos=epos, entry_mass=emass, err_flag=err)
    assert int(err) == 0
    touched = torch.zeros_like(epos, dtype=torch.bool)
    k, v, out = h.k.cpu(), h.v.cpu(), out.view(T, n_q, hd).cpu()
    bk, bv = before_k.cpu(), before_v.cpu()
    for s, a, m, n in c.spans():
        for i in range(m):
            t, e = a + i, n - m + i
            want, tol = ref.rope(qkv[t, :n_q], int(pos[t]), inv.tolist(), gq, 1e-6, inter)
            close(out[t], want, tol, f"query {t}")
            want, tol = ref.rope(qkv[t, n_q:n_q + n_kv], int(pos[t]), inv.tolist(), gk, 1e-6, inter)
            p, r = c.entry(s, e)
            close(k[p, :, r], want, tol, f"key {t}")
            assert torch.equal(v[p, :, r], qkv[t, n_q + n_kv:])
            assert bool((epos[s, :, e] == int(pos[t])).all()) and bool((emass[s, :, e] == 0).all())
            touched[s, :, e] = True
            bk[p, :, r], bv[p, :, r] = k[p, :, r], v[p, :, r]
    # nothing else was written (compared as bits: the pool holds NaN)
    assert torch.equal(k.view(torch.int16), bk.view(torch.int16))
    assert torch.equal(v.view(torch.int16), bv.view(torch.int16))
    assert bool((epos[~touched] == -9).all()) and bool((emass[~touched] == 4.0).all())


def test_rope_append_refused_entries():
    """Tokens without a place (bad page, more tokens than entries, no sequence)
    leave the cache alone; the first two raise the flag and keep their query."""
    hd, n_q, n_kv, page = 64, 2, 1, 16
    c = ref.make_cache(5, [(3, 1), (1, 20)], n_kv, hd, page)
    c.table[1, 1] = -4
    T = 6                                          # rows 4 and 5 belong to nobody
    qkv = queries(5, T, n_q + 2 * n_kv, hd).view(T, -1).cuda()
    h = handle(c)
    k0 = h.k.clone()
    out = torch.full((T, n_q * hd), 8.0, dtype=torch.float16, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    q.qk_norm_rope_append(h, qkv, c.q_start.cuda(), torch.arange(T, dtype=torch.int32).cuda(),
                          q_out=out, err_flag=err)
    assert int(err) == 1
    assert torch.equal(out[:4], qkv[:4, :n_q * hd]) and bool((out[4:] == 8.0).all())
    p, r = c.entry(0, 0)                           # the third token of sequence 0 is its only entry
    k0[p, :, r] = qkv[2, n_q * hd:(n_q + n_kv) * hd].view(n_kv, hd)
    assert torch.equal(h.k.view(torch.int16), k0.view(torch.int16))


EVICT = [
    # hd, page, n_kv, lengths, keep, sink, recent, kind of mass
    (128, 16, 2, [40], 16, 0, 0, "random"),
    (64, 16, 1, [5, 0, 17, 33], 17, 2, 4, "random"),
    (128, 32, 3, [1025, 999, 31], 500, 4, 100, "ties"),
    (64, 64, 2, [2000], 1, 0, 1, "random"),
    (128, 16, 1, [300, 301], 299, 0, 0, "equal"),
    (64, 128, 8, [777], 400, 300, 100, "odd"),
    (64, 16, 1, [5000, 4097], 4096, 4, 32, "ties"),
    (128, 256, 2, [600], 1000, 1, 1, "random"),
    (64, 256, 2, [700, 90], 60, 3, 9, "wide"),   # a table for 80,000 entries: keys made anew
    (64, 16, 4, [(37 * i) % 120 + 20 for i in range(40)], 50, 2, 8, "ties"),  # 160 heads
]


@pytest.mark.parametrize("case", range(len(EVICT)))
def test_evict(case):
    hd, page, n_kv, lens, keep, sink, recent, kind = EVICT[case]
    c = ref.make_cache(case, [(0, n) for n in lens], n_kv, hd, page, poison=False,
                       extra_pages=310 if kind == "wide" else 1)
    S, g = len(lens), torch.Generator().manual_seed(case)
    mass = torch.rand(S, n_kv, c.cap, generator=g) * 10
    if kind == "ties":
        mass = torch.floor(mass) / 2
    elif kind == "equal":
        mass[:] = 0.25
    elif kind == "odd":
        mass[:, :, ::3] = float("nan")
        mass[:, :, 1::7] = float("inf")
        mass[:, :, 2::5] = -0.0
        mass[:, :, 3::5] = 0.0
        mass[:, :, 4::5] *= -1e-40
    pos = torch.argsort(torch.rand(S, n_kv, c.cap, generator=g), -1).int()
    nxt = torch.tensor([n + 3 for n in lens], dtype=torch.int32)
    h = handle(c)
    k0, v0, n0 = h.k.clone(), h.v.clone(), h.kv_len.clone()
    md, pd = mass.cuda(), pos.cuda()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    mo = torch.full_like(md, -3.0)
    po = torch.full_like(pd, -3)
    kept, mo, po, left = q.cache_evict(h, md, pd, nxt.cuda(), keep, n_sink=sink, n_recent=recent,
                                       mass_out=mo, pos_out=po, err_flag=err)
    want, want_left = ref.evict(c, mass, pos, nxt, keep, sink, recent)
    assert left.tolist() == want_left and int(err) == 0
    assert torch.equal(kept.cpu(), want)
    assert torch.equal(h.kv_len, n0)
    for s in range(S):
        n = want_left[s]
        for hh in range(n_kv):
            src = want[s, hh, :n].long()
            assert np.array_equal(mo[s, hh, :n].cpu().numpy().view(np.int32),
                                  mass[s, hh, src].numpy().view(np.int32))
            assert torch.equal(po[s, hh, :n].cpu(), pos[s, hh, src])
            assert bool((mo[s, hh, n:] == -3.0).all()) and bool((po[s, hh, n:] == -3).all())
            for i in (src != torch.arange(n)).nonzero().view(-1).tolist():
                (pa, ra), (pb, rb) = c.entry(s, int(src[i])), c.entry(s, i)
                k0[pb, hh, rb], v0[pb, hh, rb] = c.k[pa, hh, ra].cuda(), c.v[pa, hh, ra].cuda()
    assert torch.equal(h.k, k0) and torch.equal(h.v, v0)


def test_evict_bad_page_is_listed_but_not_copied():
    c = ref.make_cache(9, [(0, 64)], 1, 64, 16, poison=False)
    c.table[0, 3] = 99                              # entries 48..63: their rows cannot be read
    mass = torch.arange(c.cap).float().view(1, 1, -1)
    pos = torch.arange(c.cap, dtype=torch.int32).view(1, 1, -1)
    h = handle(c)
    k0 = h.k.clone()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    kept, *_ = q.cache_evict(h, mass.cuda(), pos.cuda(), torch.tensor([64], dtype=torch.int32).cuda(),
                             16, err_flag=err)
    assert int(err) == 1 and kept.view(-1).tolist() == list(range(48, 64))
    assert torch.equal(h.k, k0)


def test_graphs_streams_and_shared_workspace():
    """Two captured graphs that share a workspace, replayed in turn on another
    stream, follow what their inputs hold at replay."""
    hd, n_q, n_kv = 128, 8, 2
    # (a cache long enough for its parts to be joined through the workspace)
    cs = [ref.make_cache(20 + i, [(1, 13000), (1, 1)], n_kv, hd, 16) for i in range(2)]
    hs = [handle(c) for c in cs]
    xs = [queries(20 + i, 2, n_q, hd).cuda() for i in range(2)]
    qs = cs[0].q_start.cuda()
    n = q.paged_attention_workspace_bytes(hs[0], 2, n_q, 1)
    assert n > 0
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    outs = [torch.zeros(2, n_q * hd, dtype=torch.float16, device="cuda") for _ in range(2)]
    lses = [torch.zeros(2, n_q, device="cuda") for _ in range(2)]
    masses = [torch.zeros(2, n_kv, c.cap, device="cuda") for c in cs]
    side, graphs = torch.cuda.Stream(), []
    side.wait_stream(torch.cuda.current_stream())
    for i in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=side):
            q.paged_attention(hs[i], xs[i], qs, max_q=1, out=outs[i], lse=lses[i], workspace=ws)
            q.attention_mass(hs[i], xs[i], qs, lses[i], max_q=1, mass_out=masses[i])
        graphs.append(gr)
    for turn in range(2):
        for i in range(2):
            xs[i].copy_(queries(40 + turn * 2 + i, 2, n_q, hd))
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            for i in (0, 1, 0):
                graphs[i].replay()
        torch.cuda.synchronize()
        for i in range(2):
            want, want_lse, tol, lse_tol = ref.attention(cs[i], xs[i].cpu(), hd ** -0.5)
            close(outs[i].view(2, n_q, hd), want, tol, "replayed out")
            close(lses[i], want_lse, lse_tol, "replayed lse")
            # the same call on a stream of its own, temporaries included
            o, _ = q.paged_attention(hs[i], xs[i], qs, max_q=1, stream=side)
            side.synchronize()
            assert torch.equal(o, outs[i])


@pytest.mark.parametrize("norm", [False, True])
def test_decode_loop(norm):
    """A layer's decoding with a budget: QKV matvec, norms + rotation + append,
    attention, its weights, eviction whenever the cache is over its budget, and
    o_proj, against the same steps in 64 bits on the operators' own fp16
    tensors.  The cache the operators keep is compared after every step."""
    H, n_q, n_kv, hd, page, keep = 1024, 8, 4, 64, 16, 24
    grp, eps = n_q // n_kv, 1e-6
    wqkv = synth.quant_weight(synth.rng(8, 0, synth.TID["qkv"]), (n_q + 2 * n_kv) * hd, H, 4)
    wo = synth.quant_weight(synth.rng(8, 0, synth.TID["o"]), 1024, n_q * hd, 4) if n_q * hd % 64 == 0 else None
    wqkv_d, wo_d = dev_weight(wqkv), dev_weight(wo)
    g = torch.Generator().manual_seed(4)
    gamma = [(1 + 0.1 * torch.randn(hd, generator=g)).half().cuda() if norm else None for _ in range(2)]
    inv = (5e5 ** (-torch.arange(0, hd, 2).double() / hd)).float()
    cap_pages = 3
    c = ref.Cache(torch.zeros(4, n_kv, page, hd).half(), torch.zeros(4, n_kv, page, hd).half(),
                  torch.tensor([[2, 0, 3]], dtype=torch.int32), torch.zeros(1, dtype=torch.int32),
                  torch.tensor([0, 1], dtype=torch.int32))
    h = handle(c)
    qs = c.q_start.cuda()
    mass = torch.zeros(1, n_kv, cap_pages * page, device="cuda")
    epos = torch.full((1, n_kv, cap_pages * page), -1, dtype=torch.int32, device="cuda")
    mass2, epos2 = torch.zeros_like(mass), torch.full_like(epos, -1)
    model = [[] for _ in range(n_kv)]              # per head: (position, mass) in cache order
    for step in range(60):
        # the weights' mean is negative: small activations keep fp16 in range
        x = (torch.randn(H, generator=g) * 0.05).half().cuda()
        qkv = q.qgemv_w4g64(wqkv_d, x)
        pos = torch.tensor([step], dtype=torch.int32, device="cuda")
        h.kv_len += 1
        qr = q.qk_norm_rope_append(h, qkv.view(1, -1), qs, pos, inv.cuda(), q_norm=gamma[0],
                                   k_norm=gamma[1], eps=eps, entry_pos=epos, entry_mass=mass)
        out, lse = q.paged_attention(h, qr, qs, max_q=1, want_lse=True)
        q.attention_mass(h, qr, qs, lse, max_q=1, mass=mass, mass_out=mass)
        y = q.qgemv_w4g64(wo_d, out[0])
        n = int(h.kv_len)
        # attention over exactly the entries the model says are there
        c.k, c.v, c.lens = h.k.cpu(), h.v.cpu(), h.kv_len.cpu()
        raw = qkv.cpu().view(n_q + 2 * n_kv, hd)
        p, r = c.entry(0, n - 1)
        want, tol = ref.rope(raw[n_q:n_q + n_kv], step, inv.tolist(),
                             None if not norm else gamma[1].cpu(), eps, False)
        close(c.k[p, :, r], want, tol, "appended key")
        assert torch.equal(c.v[p, :, r], raw[n_q + n_kv:])
        want, _, tol, _ = ref.attention(c, qr.cpu().view(1, n_q, hd), hd ** -0.5)
        close(out.view(1, n_q, hd), want, tol, "out")
        assert bool(torch.isfinite(y).all())
        for hh in range(n_kv):
            model[hh].append(step)
            assert epos[0, hh, :n].tolist() == model[hh]
        if n > 30:
            kept, _, _, left = q.cache_evict(h, mass, epos, pos + 1, keep, n_sink=2, n_recent=6,
                                             mass_out=mass2, pos_out=epos2)
            want, _ = ref.evict(c, mass.cpu(), epos.cpu(), (pos + 1).cpu(), keep, 2, 6)
            assert torch.equal(kept.cpu(), want)
            for hh in range(n_kv):
                model[hh] = [model[hh][i] for i in want[0, hh].tolist()]
                assert {0, 1} <= set(model[hh]) and set(range(step - 5, step + 1)) <= set(model[hh])
            mass, mass2, epos, epos2 = mass2, mass, epos2, epos
            h.kv_len.copy_(left)
    assert grp == 2 and q.device_status() == 0


@pytest.mark.parametrize("m,n_q", [(2, 4), (40, 8)])
def test_workspace_off_a_32_byte_boundary(m, n_q):
    """A workspace needs 16 bytes of alignment, not more."""
    c = ref.make_cache(3, [(m, 13000)], 2, 64, 16)
    x, h, qs = queries(3, m, n_q, 64).cuda(), handle(c), c.q_start.cuda()
    n = q.paged_attention_workspace_bytes(h, m, n_q, m)
    assert n > 0
    whole = torch.empty(n + 16, dtype=torch.uint8, device="cuda")
    out, lse = q.paged_attention(h, x, qs, max_q=m, want_lse=True)
    out1, lse1 = q.paged_attention(h, x, qs, max_q=m, want_lse=True, workspace=whole[16:])
    assert torch.equal(out, out1) and torch.equal(lse, lse1)


@pytest.mark.parametrize("n_q,m", [(4, 2), (8, 8)])
def test_longest_cache(n_q, m):
    """2^29 entries of one head (a page table that repeats a page of zero keys,
    and a last page of its own): the four calls in a row, at the ends of
    every 32-bit product of entries, rows and bytes."""
    hd, page, cap, w = 64, 256, 1 << 29, 20.0
    g = torch.Generator().manual_seed(n_q)
    k = torch.zeros(2, 1, page, hd, dtype=torch.float16)
    k[1, 0, :, 0] = w                                     # weight e^w against 1
    v = torch.randint(-4, 5, (2, 1, page, hd), generator=g).half()
    table = torch.zeros(1, cap // page, dtype=torch.int32)
    table[0, -1] = 1
    h = q.kv_cache(k.cuda(), v.cuda(), table.cuda(), torch.tensor([cap], dtype=torch.int32).cuda())
    qkv = torch.zeros(m, n_q + 2, hd, dtype=torch.float16)
    qkv[:, :n_q, 0] = 1.0
    qkv[:, n_q, 0] = w
    qkv[:, n_q + 1] = torch.randint(-4, 5, (m, hd), generator=g).half()
    v[1, 0, page - m:] = qkv[:, n_q + 1]
    mass = torch.full(h.entries, 9.0, device="cuda")
    pos = torch.zeros(h.entries, dtype=torch.int32, device="cuda")
    qs = torch.tensor([0, m], dtype=torch.int32, device="cuda")
    at = torch.arange(cap - m, cap, dtype=torch.int32)
    x = q.qk_norm_rope_append(h, qkv.view(m, -1).cuda(), qs, at.cuda(), entry_pos=pos, entry_mass=mass)
    assert torch.equal(x.cpu(), qkv[:, :n_q].reshape(m, -1)) and torch.equal(h.v.cpu(), v)
    assert torch.equal(h.k.cpu(), k)
    assert torch.equal(pos[0, 0, -m:].cpu(), at) and int(pos.count_nonzero()) == m
    assert int(mass.count_nonzero()) == cap - m
    out, lse = q.paged_attention(h, x, qs, max_q=m, scale=1.0, want_lse=True)
    # exact sums: page 0 as often as the table has it, then the last page's rows
    V0, V1, heavy = v[0, 0].double(), v[1, 0].double(), math.exp(w)
    for i in range(m):
        n1 = page - m + i + 1
        total = (cap - page) + heavy * n1
        want = ((cap // page - 1) * V0.sum(0) + heavy * V1[:n1].sum(0)) / total
        # fp32 exponents of up to 29 (2^-20), the sums, and one rounding to fp16
        assert torch.allclose(out[i].view(n_q, hd).cpu().double(), want.expand(n_q, hd),
                              rtol=2.0 ** -11 + 1e-5, atol=1e-5)
        assert torch.allclose(lse[i].cpu().double(), torch.tensor(math.log(total)).double(), atol=1e-5)
    mass.zero_()
    q.attention_mass(h, x, qs, lse, max_q=m, scale=1.0, mass=mass, mass_out=mass)
    low = float(torch.exp(-lse.double()).sum())           # what every entry of weight 1 receives
    first = mass[0, 0, :cap - page]
    # exponents up to 42: 2^-19 relative to the weight, with those of lse
    assert float(first.min()) >= low * (1 - 2e-5) and float(first.max()) <= low * (1 + 2e-5)
    for j in (cap - page, cap - m - 1, cap - m, cap - 1):
        want = float(torch.exp(w - lse[max(0, j - (cap - m)):].double()).sum())
        assert abs(float(mass[0, 0, j]) - want) <= 2e-5 * want
    # eviction: the lightest five go, the last five entries take their places
    pos = torch.arange(cap, dtype=torch.int32, device="cuda").view(1, 1, -1)
    out_of = torch.tensor([3, 1 << 20, (1 << 28) + 1, (1 << 28) + 77777, cap - 300])
    mass[0, 0, out_of.cuda()] = 0.0
    keep = cap - 5
    kept, mass1, pos1, n = q.cache_evict(h, mass, pos, torch.tensor([cap], dtype=torch.int32).cuda(), keep)
    assert n.tolist() == [keep]
    want = torch.arange(keep, dtype=torch.int32, device="cuda")
    want[out_of.cuda()] = torch.arange(keep, cap, dtype=torch.int32, device="cuda")
    assert torch.equal(kept[0, 0], want) and torch.equal(pos1[0, 0, :keep], want)
    assert torch.equal(mass1[0, 0, :keep], mass[0, 0, want.long()])
    # the rows moved: on page 0, which every sequence of holes shares, in the last ones' order
    moved = {int(j) % page: keep + i - (cap - page) for i, j in enumerate(out_of.tolist())}
    for r, src in moved.items():
        assert torch.equal(h.v[0, 0, r].cpu(), v[1, 0, src])


@pytest.mark.parametrize("m,ws", [(2, True), (40, True), (40, False)])
def test_hidden_nan_behind_a_long_cache(m, ws):
    """All rows but the last token's are computed again without the NaN that it
    alone sees, over a cache long enough for that to take a while."""
    hd, n_kv, n_q, n = 64, 1, 8, 20000
    c = ref.make_cache(11, [(m, n)], n_kv, hd, 64)
    x = queries(11, m, n_q, hd)
    want, _, tol, _ = ref.attention(c, x, hd ** -0.5)
    p, r = c.entry(0, n - 1)
    c.v[p, :, r] = math.nan
    w0 = None if ws else torch.empty(0, dtype=torch.uint8, device="cuda")
    q.device_status()
    out, _ = q.paged_attention(handle(c), x.cuda(), c.q_start.cuda(), max_q=m, workspace=w0)
    out = out.view(m, n_q, hd)
    close(out[:m - 1], want[:m - 1], tol[:m - 1], "rows before the NaN")
    assert bool(torch.isnan(out[m - 1]).all()) and q.device_status() == 0
