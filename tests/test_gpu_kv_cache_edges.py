"""Rare inputs of the paged-cache operators: rows that the caller masks, weights far below
a row's largest, positions at the end of the 32-bit range, starts and lengths out of range
where no token lies."""
import math

import pytest
import torch

import kv_reference as ref
from test_gpu_kv_cache import close, handle, queries

pytestmark = pytest.mark.gpu

q = pytest.importorskip("bit_group_quantized_qgemv_gb300")


@pytest.mark.parametrize("value", [math.nan, math.inf])
@pytest.mark.parametrize("n_q,n_kv,m", [(4, 1, 5), (8, 1, 4), (4, 4, 20), (4, 1, 20), (6, 2, 40), (2, 2, 200),
                                        (8, 1, 90), (160, 1, 2)])
def test_rows_of_no_lse_add_nothing(n_q, n_kv, m, value):
    """A row whose lse is -inf adds nothing, whatever its query holds."""
    hd, n = 64, 300
    c = ref.make_cache(m, [(m, n), (1, 40)], n_kv, hd, 16)
    x = queries(m, m + 1, n_q, hd)
    _, lse, _, _ = ref.attention(c, x, hd ** -0.5)
    lse = lse.float()
    masked = [0, m // 2, m - 1]
    lse[masked] = -math.inf
    lse[1, n_q - 1] = -math.inf                     # one head of a token that counts otherwise
    mass = torch.rand(2, n_kv, c.cap)
    want, tol = ref.attention_mass(c, x, lse, hd ** -0.5, mass)
    x[masked] = value
    x[1, n_q - 1] = value
    got = q.attention_mass(handle(c), x.cuda(), c.q_start.cuda(), lse.cuda(), max_q=m, mass=mass.cuda())
    close(got[0, :, :n], want[0, :, :n], tol[0, :, :n], "mass")
    close(got[1, :, :40], want[1, :, :40], tol[1, :, :40], "mass of the other sequence")
    assert q.device_status() == 0


@pytest.mark.parametrize("rows", [(1, 1), (6, 4), (75, 4)])   # new tokens, query heads
@pytest.mark.parametrize("n,at", [(3000, 0), (14000, 0), (3000, 1500)])
@pytest.mark.parametrize("nats", [12.3, 16.7, 18.0, 19.5])
def test_light_entries_next_to_a_heavy_one(rows, n, at, nats):
    """One entry of weight 1 with values of zero, all others e^-nats with values of one sign:
    the output is what the light ones add up to.

    A weight is rounded to fp16 (2^-11 of it, or 2^-32 of the largest weight), the exponent
    errs by 2^-22 (nats + 1), the output by half a step of fp16 (2^-11, or 2^-25).  The sum of
    the weights is one of fp32 additions: equal light weights onto a heavy one are all rounded
    the same way, each by up to half a unit of the sum, 2^-24 of it.  The fewest
    threads that share a row's entries are 4 warps of 8, so one adds up to n / 32 of them, and
    40 more additions join the threads, warps and blocks: (n / 32 + 40) 2^-24 of the sum, which
    is as much of the output and, in nats, of lse.  (The many-rows kernel adds 128 entries at a
    time: n / 128.)"""
    m, n_q = rows
    hd, page = 64, 64
    c = ref.make_cache(n + m, [(m, n)], 1, hd, page)
    g = torch.Generator().manual_seed(m)
    value = (1000 * (0.5 + torch.rand(n, hd, generator=g))).half()
    heavy = torch.tensor(nats).half()
    value[at] = 0
    for e in range(0, n, page):
        p, _ = c.entry(0, e)
        k = min(page, n - e)
        c.k[p, 0, :k, 0] = 0
        c.v[p, 0, :k] = value[e:e + k]
    p, r = c.entry(0, at)
    c.k[p, 0, r, 0] = heavy
    x = torch.zeros(m, n_q, hd).half()
    x[:, :, 0] = 1
    light = math.exp(-float(heavy))
    added = (n / 32 + 40) * 2.0 ** -24
    sums = torch.cumsum(value.double(), 0)
    none = torch.empty(0, dtype=torch.uint8, device="cuda")
    for ws in (None, none):
        out, lse = q.paged_attention(handle(c), x.cuda(), c.q_start.cuda(), max_q=m, scale=1.0, want_lse=True,
                                     workspace=ws)
        for i in range(m):
            e = n - m + i                           # sees the heavy entry and e light ones
            z = 1 + e * light
            want = (light * sums[e] / z).expand(n_q, hd)
            tol = (want * (2.0 ** -10 + 2.0 ** -21 * (nats + 1) + added) + 2.0 ** -32 * sums[e] / z + 2.0 ** -25)
            close(out[i].view(n_q, hd), want, tol, f"row {i}")
            close(lse[i], torch.full((n_q,), float(heavy) + math.log(z)).double(),
                  torch.full((n_q,), 2.0 ** -21 * (nats + 1) + added).double(), f"lse {i}")
    assert q.device_status() == 0


PI_60 = 3141592653589793238462643383279502884197169399375105820974944   # pi 10^60
TURN = (10 ** 60 << 192) // (2 * PI_60)                                 # 2^192 / (2 pi)


def test_rotation_of_far_positions():
    """Positions at both ends of int32 at which a sine or a cosine is close to 0: the angle has
    to be right to 3e-6 (as kv_reference.rope allows, which takes it from a rounded product)."""
    hd, page, T = 64, 256, 256
    at = list(range(2 ** 31 - 300000, 2 ** 31)) + list(range(-2 ** 31, -2 ** 31 + 300000))
    # how far position * 1 is from a whole number of quarter turns, in 2^-64 of them
    quarter = ((p, (4 * p * TURN >> 128) + (1 << 63) & (1 << 64) - 1) for p in at)
    near = [p for p, x in quarter if abs(x - (1 << 63)) < (1 << 64) // 4000]
    pos = (near + at[:T])[:T]
    assert len(near) > T // 2
    inv = torch.ones(hd // 2)
    inv[1::2] = torch.rand(hd // 4, generator=torch.Generator().manual_seed(1))
    qkv = torch.zeros(T, 3, hd).half()
    qkv[:, :, :hd // 2] = 1.0
    k = torch.zeros(1, 1, page, hd).half().cuda()
    h = q.kv_cache(k, k.clone(), torch.zeros(1, 1, dtype=torch.int32).cuda(),
                   torch.tensor([T], dtype=torch.int32).cuda())
    out = q.qk_norm_rope_append(h, qkv.view(T, -1).cuda(), torch.tensor([0, T], dtype=torch.int32).cuda(),
                                torch.tensor(pos, dtype=torch.int32).cuda(), inv.cuda())
    # a float is a whole number over 2^149; the turn is taken from 2^64 parts of it
    num = [int(f.double().item() * 2 ** 149) for f in inv]
    turn = torch.tensor([[((p * n * TURN >> 277) & (1 << 64) - 1) / 2 ** 64 for n in num] for p in pos],
                        dtype=torch.float64)
    want = torch.cat([torch.cos(2 * math.pi * turn), torch.sin(2 * math.pi * turn)], 1)
    tol = 2.0 ** -11 * want.abs() + 3e-6 + 2.0 ** -25
    close(out, want, tol, "queries")
    close(h.k[0, 0], want, tol, "keys")


@pytest.mark.parametrize("starts,lens", [
    ([0, 5, 3, 8], [20, 20, 20]),                   # falls where no token looks
    ([0, 8, 8, 6], [20, 20, 20]),
    ([0, 0, 4, 8], [-1, 20, 20]),                   # lengths of sequences without new tokens
    ([0, 8, 8, 8], [20, 20, 33]),
    ([0] * 200 + [8, 8], [20] * 199 + [20, 999]),
])
def test_rope_append_looks_at_every_sequence(starts, lens):
    hd, T, S = 64, 8, len(lens)
    k = torch.zeros(2 * S, 1, 16, hd).half().cuda()
    table = torch.arange(2 * S, dtype=torch.int32).view(S, 2).cuda()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    qkv = queries(1, T, 3, hd).cuda().view(T, -1)
    pos = torch.arange(T, dtype=torch.int32).cuda()
    good = torch.tensor([0] * S + [T], dtype=torch.int32).cuda()
    q.qk_norm_rope_append(q.kv_cache(k, k.clone(), table, torch.full((S,), 20, dtype=torch.int32).cuda()),
                          qkv, good, pos, err_flag=err)
    assert int(err) == 0
    h = q.kv_cache(k, k.clone(), table, torch.tensor(lens, dtype=torch.int32).cuda())
    q.qk_norm_rope_append(h, qkv, torch.tensor(starts, dtype=torch.int32).cuda(), pos, err_flag=err)
    assert int(err) == 1


@pytest.mark.parametrize("n_q", [2, 64])
@pytest.mark.parametrize("starts,lens,max_q", [
    ([0, 2, 1, 1], [20, 0, 20], 2),                 # the one that falls has no entries
    ([0, 1, 1, 9], [20, 20, 0], 2),
    ([0, 0, 2, 2], [20, 0, 20], 1),                 # more tokens than declared, without entries
    ([0] * 100 + [2, 2], [20] * 99 + [0, 20], 1),
])
def test_mass_looks_at_every_sequence(starts, lens, max_q, n_q):
    hd, T, S = 64, 2, len(lens)
    k = torch.zeros(2 * S, 1, 16, hd).half().cuda()
    table = torch.arange(2 * S, dtype=torch.int32).view(S, 2).cuda()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    x = queries(1, T, n_q, hd).cuda()
    lse = torch.zeros(T, n_q).cuda()
    h = q.kv_cache(k, k.clone(), table, torch.tensor(lens, dtype=torch.int32).cuda())
    q.attention_mass(h, x, torch.tensor([0] * S + [1], dtype=torch.int32).cuda(), lse, max_q=max_q, err_flag=err)
    assert int(err) == 0
    q.attention_mass(h, x, torch.tensor(starts, dtype=torch.int32).cuda(), lse, max_q=max_q, err_flag=err)
    assert int(err) == 1


def off(t, by=1):
    """The same tensor on the GPU, `by` elements behind an aligned address."""
    buf = torch.empty(t.numel() + by, dtype=t.dtype, device="cuda")
    view = buf[by:].view(t.shape)
    view.copy_(t)
    return view


@pytest.mark.parametrize("hd,n_q,n_kv,seqs", [(64, 3, 1, [(1, 500), (2, 77)]), (128, 8, 2, [(40, 300), (1, 9)])])
def test_numbers_off_their_16_byte_boundaries(hd, n_q, n_kv, seqs):
    """Starts, lengths, lse and mass need 4 bytes of alignment, the fused QKV rows 8 and
    strides that are multiples of 4."""
    c = ref.make_cache(7, seqs, n_kv, hd, 16)
    T, max_q, scale = sum(m for m, _ in seqs), max(m for m, _ in seqs), hd ** -0.5
    x = queries(7, T, n_q, hd)
    h = q.kv_cache(c.k.cuda(), c.v.cuda(), off(c.table), off(c.lens, 3))
    qs = off(c.q_start)
    want, want_lse, tol, lse_tol = ref.attention(c, x, scale)
    out, lse = q.paged_attention(h, x.cuda(), qs, max_q=max_q, lse=off(torch.zeros(T, n_q)))
    close(out.view(T, n_q, hd), want, tol, "out")
    close(lse, want_lse, lse_tol, "lse")
    mass = torch.rand(len(seqs), n_kv, c.cap)
    got = q.attention_mass(h, x.cuda(), qs, lse, max_q=max_q, mass=off(mass), mass_out=off(torch.zeros_like(mass), 2))
    want_m, tol_m = ref.attention_mass(c, x, lse.cpu(), scale, mass)
    for s, (_, n) in enumerate(seqs):
        close(got[s, :, :n], want_m[s, :, :n], tol_m[s, :, :n], "mass")
    # QKV rows behind four values, 4 values apart; queries into rows like that
    w = (n_q + 2 * n_kv) * hd
    wide = torch.zeros(T * (w + 4) + 4).half().cuda()[4:].view(T, w + 4)
    qkv = queries(8, T, n_q + 2 * n_kv, hd).view(T, w)
    wide[:, :w] = qkv.cuda()
    room = torch.zeros(T * (n_q * hd + 12) + 4).half().cuda()[4:].view(T, n_q * hd + 12)
    pos = off(torch.arange(T, dtype=torch.int32))
    inv = off(torch.rand(hd // 2))
    gamma = torch.rand(hd).half()
    q.qk_norm_rope_append(h, wide[:, :w], qs, pos, inv, q_norm=off(gamma, 4), k_norm=off(gamma, 4),
                          q_out=room[:, :n_q * hd], entry_mass=off(mass))
    for t in range(T):
        want, tol = ref.rope(qkv[t].view(-1, hd)[:n_q], t, inv.tolist(), gamma, 1e-6, False)
        close(room[t, :n_q * hd].view(n_q, hd), want, tol, "query")
    assert bool((room[:, n_q * hd:] == 0).all())


@pytest.mark.parametrize("n_kv,lens,keep,extra", [(2, [700, 40], 300, 0), (8, [300] * 24, 200, 0),
                                                  (2, [700, 90], 60, 3300)])
def test_evict_off_16_byte_boundaries(n_kv, lens, keep, extra):
    c = ref.make_cache(3, [(0, n) for n in lens], n_kv, 64, 16, poison=False, extra_pages=extra)
    S, g = len(lens), torch.Generator().manual_seed(3)
    mass = torch.floor(torch.rand(S, n_kv, c.cap, generator=g) * 40)
    pos = torch.argsort(torch.rand(S, n_kv, c.cap, generator=g), -1).int()
    nxt = torch.tensor(lens, dtype=torch.int32)
    kept, mo, po, left = q.cache_evict(
        handle(c), off(mass), off(pos, 2), off(nxt), keep, n_sink=3, n_recent=8,
        kept=off(torch.zeros(S, n_kv, keep, dtype=torch.int32), 3), mass_out=off(torch.zeros_like(mass), 3),
        pos_out=off(torch.zeros_like(pos)), kv_len_out=off(torch.zeros(S, dtype=torch.int32), 2))
    want, want_left = ref.evict(c, mass, pos, nxt, keep, 3, 8)
    assert left.tolist() == want_left and torch.equal(kept.cpu(), want)
    for s, n in enumerate(want_left):
        for hh in range(n_kv):
            src = want[s, hh, :n].long()
            assert torch.equal(mo[s, hh, :n].cpu(), mass[s, hh, src])
            assert torch.equal(po[s, hh, :n].cpu(), pos[s, hh, src])


@pytest.mark.parametrize("n_q,n_kv,seqs", [(2, 2, [(50, 0)]), (4, 1, [(60, 0), (9, 9), (300, 2), (0, 40)]),
                                           (6, 2, [(30, 7)] * 40)])
def test_many_new_tokens_over_empty_caches(n_q, n_kv, seqs):
    hd = 64
    c = ref.make_cache(1, seqs, n_kv, hd, 16)
    T, max_q = sum(m for m, _ in seqs), max(m for m, _ in seqs)
    x = queries(1, T, n_q, hd)
    want, want_lse, tol, lse_tol = ref.attention(c, x, hd ** -0.5)
    for ws in (None, torch.empty(0, dtype=torch.uint8, device="cuda")):
        out = torch.full((T, n_q, hd), 5.0).half().cuda()
        _, lse = q.paged_attention(handle(c), x.cuda(), c.q_start.cuda(), max_q=max_q, out=out, want_lse=True,
                                   workspace=ws)
        close(out, want, tol, "out")
        close(lse, want_lse, lse_tol, "lse")
    m = q.attention_mass(handle(c), x.cuda(), c.q_start.cuda(), lse, max_q=max_q)
    want_m, tol_m = ref.attention_mass(c, x, lse.cpu(), hd ** -0.5, torch.zeros(len(seqs), n_kv, c.cap))
    close(m, want_m, tol_m, "mass")
    assert q.device_status() == 0


def test_calls_on_two_streams_at_once():
    """Calls of every kernel on two streams, workspaces of their own: as one after the other."""
    jobs = []
    for i, (n_q, seqs) in enumerate([(4, [(1, 9000), (1, 5000)]), (8, [(60, 3000)]), (4, [(1, 14000)]),
                                     (2, [(200, 700)]), (4, [(7, 4000)] * 4)]):
        c = ref.make_cache(70 + i, seqs, 2, 64, 16)
        T, m = sum(m for m, _ in seqs), max(m for m, _ in seqs)
        jobs.append((handle(c), queries(70 + i, T, n_q, 64).cuda(), c.q_start.cuda(), m))

    def run(job):
        h, x, qs, m = job
        out, lse = q.paged_attention(h, x, qs, max_q=m, want_lse=True)
        return out, lse, q.attention_mass(h, x, qs, lse, max_q=m)

    want = [run(j) for j in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for turn in range(4):
        for k, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[k] += [(i, run(jobs[i])) for i in (range(5) if k == 0 else reversed(range(5)))]
    torch.cuda.synchronize()
    for i, res in got[0] + got[1]:
        assert all(torch.equal(a, b) for a, b in zip(res, want[i]))
    assert q.device_status() == 0


@pytest.mark.parametrize("rows", [(1, 1), (6, 4), (75, 4)])
@pytest.mark.parametrize("size", [256, 2048, 4096, 5120, 7168])
def test_large_scores_that_grow(rows, size):
    """Scores of up to 5 10^7 whose maximum grows a little from tile to tile, at which floats
    lie up to 4 apart: whatever the weights then are, they add up to 1 (two roundings to
    fp16, of a weight and of the output), and no weight leaves fp16's range."""
    m, n_q = rows
    hd, page, n = 64, 16, 1500
    for step in range(1, 14):
        c = ref.make_cache(m, [(m, n)], 1, hd, page)
        c.v[torch.isfinite(c.v)] = 1.0
        for e in range(0, n, page):
            p, _ = c.entry(0, e)
            k = min(page, n - e)
            c.k[p, 0, :k] = 0
            c.k[p, 0, :k, 0] = size
            c.k[p, 0, :k, 1] = (e // 128) * step / 2    # (a tile of 128, and the warps' four of 16)
        x = torch.zeros(m, n_q, hd).half()
        x[:, :, 0] = size
        x[:, :, 1] = 1
        for ws in (None, torch.empty(0, dtype=torch.uint8, device="cuda")):
            out, lse = q.paged_attention(handle(c), x.cuda(), c.q_start.cuda(), max_q=m, scale=1.0, want_lse=True,
                                         workspace=ws)
            one = torch.ones(m, n_q * hd, dtype=torch.float64)
            close(out, one, 2.0 ** -10 * one, f"step {step}")
            assert bool(torch.isfinite(lse).all())
