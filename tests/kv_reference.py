"""Plain 64-bit forms of the paged-cache operators, on the CPU, and the
inputs the tests feed them.  Shares nothing with the CUDA path."""
import math
from dataclasses import dataclass

import numpy as np
import torch


@dataclass
class Cache:
    k: torch.Tensor
    v: torch.Tensor
    table: torch.Tensor
    lens: torch.Tensor
    q_start: torch.Tensor

    @property
    def page(self):
        return self.k.shape[2]

    @property
    def cap(self):
        return self.table.shape[1] * self.page

    def entry(self, s, i):
        """(page, row) of entry i of sequence s; page None when it is bad."""
        p = int(self.table[s, i // self.page])
        return (p if 0 <= p < self.k.shape[0] else None), i % self.page

    def rows(self, s, n, pool):
        """Entries 0..n-1 of sequence s in float64 [n][n_kv][hd] and which are on good pages."""
        out = torch.zeros(n, pool.shape[1], pool.shape[3], dtype=torch.float64)
        good = torch.zeros(n, dtype=torch.bool)
        for i in range(0, n, self.page):
            p, _ = self.entry(s, i)
            m = min(self.page, n - i)
            if p is not None:
                out[i:i + m] = pool[p, :, :m].transpose(0, 1).double()
                good[i:i + m] = True
        return out, good

    def spans(self):
        """(sequence, first row, new tokens, length) with the documented clamps."""
        for s in range(len(self.lens)):
            a, b = int(self.q_start[s]), int(self.q_start[s + 1])
            yield s, a, b - a, int(self.lens[s])


def make_cache(seed, seqs, n_kv, hd, page, spare=2, extra_pages=1, poison=True):
    """seqs: list of (new tokens, length).  Everything in the pool that no
    sequence owns, the rows behind each length included, is NaN or inf."""
    g = torch.Generator().manual_seed(seed)
    need = [(n + page - 1) // page for _, n in seqs]
    n_pages = sum(need) + spare
    order = torch.randperm(n_pages, generator=g).int()
    table = torch.full((len(seqs), max(need + [1]) + extra_pages), int(order[-1]), dtype=torch.int32)
    k = torch.full((n_pages, n_kv, page, hd), float("nan") if poison else 0.0).half()
    v = k.clone()
    if poison:
        v[:, :, ::2] = float("inf")
    at = 0
    for s, (_, n) in enumerate(seqs):
        table[s, :need[s]] = order[at:at + need[s]]
        for i in range(0, n, page):
            m = min(page, n - i)
            p = int(order[at + i // page])
            k[p, :, :m] = torch.randn(n_kv, m, hd, generator=g).half()
            v[p, :, :m] = torch.randn(n_kv, m, hd, generator=g).half()
        at += need[s]
    q_start = torch.tensor(np.cumsum([0] + [q for q, _ in seqs]), dtype=torch.int32)
    return Cache(k, v, table, torch.tensor([n for _, n in seqs], dtype=torch.int32), q_start)


def attention(c, q, scale):
    """out, lse and the tolerances of both (float64).  q: fp16 [T][n_q][hd].

    Scores: the tensor cores' fp32 sums were measured at 9.1e-7 of sum |a b|
    per product of 16, so 8 of them err by at most d = 8e-6 scale sum |q k|.
    That moves every weight by at most a factor e^(+-2d) (its own score and the
    maximum's); weights are rounded to fp16 (half a step 2^-11, below 2^-14 at
    most 2^-25 absolute against a largest weight of 1), ex2 and the fp32 sums
    add 4e-6; the output is rounded once (2^-11)."""
    T, n_q, hd = q.shape
    out = torch.zeros(T, n_q, hd, dtype=torch.float64)
    tol = torch.full_like(out, 1e-7)
    lse = torch.full((T, n_q), -math.inf, dtype=torch.float64)
    lse_tol = torch.full((T, n_q), 1e-7, dtype=torch.float64)
    grp = n_q // c.k.shape[1]
    for s, a, m, n in c.spans():
        K, good = c.rows(s, n, c.k)
        V, _ = c.rows(s, n, c.v)
        for i in range(m):
            see = good & (torch.arange(n) <= n - m + i)
            if not bool(see.any()):
                continue
            for h in range(n_q):
                kk, vv = K[see][:, h // grp], V[see][:, h // grp]
                x = q[a + i, h].double()
                sc = kk @ x * scale
                d = 8e-6 * scale * float((kk.abs() @ x.abs()).max())
                w = torch.exp(sc - sc.max())
                z = w.sum()
                o = (w @ vv) / z
                out[a + i, h] = o
                lse[a + i, h] = sc.max() + torch.log(z)
                tol[a + i, h] = (2.0 ** -11 * o.abs() + (w @ vv.abs()) / z * (2.0 ** -11 + 2 * d + 4e-6)
                                 + 2.0 ** -25 * vv.abs().sum(0) / z + 2.0 ** -25)
                lse_tol[a + i, h] = d + 4e-6 + 2.0 ** -22 * abs(float(lse[a + i, h]))
    return out, lse, tol, lse_tol


def attention_mass(c, q, lse, scale, mass):
    """mass plus the weights, and the tolerance: each weight by its score's
    error d (as above) and the fp32 roundings of the exponent (2^-22 of its two
    terms), the sum by one rounding per row."""
    T, n_q, hd = q.shape
    n_kv = c.k.shape[1]
    grp = n_q // n_kv
    out, tol = mass.double().clone(), torch.full(mass.shape, 1e-9, dtype=torch.float64)
    for s, a, m, n in c.spans():
        K, good = c.rows(s, n, c.k)
        for h in range(n_q):
            for i in range(m):
                see = good & (torch.arange(n) <= n - m + i)
                L = float(lse[a + i, h])
                if L == -math.inf:
                    continue
                x = q[a + i, h].double()
                sc = K[:, h // grp] @ x * scale
                w = torch.where(see, torch.exp(sc - L), 0.0)
                d = 8e-6 * scale * (K[:, h // grp].abs() @ x.abs()) + 2.0 ** -22 * (sc.abs() + abs(L) + 4)
                out[s, h // grp, :n] += w
                tol[s, h // grp, :n] += torch.where(see, w * d, 0.0)
        tol[s, :, :n] += (m * grp + 2) * 2.0 ** -24 * out[s, :, :n].abs()
    return out, tol


def rope(x, pos, inv_freq, gamma, eps, inter):
    """x fp16 [heads][hd] of one token -> float64 and its tolerance (fp32
    arithmetic of a few roundings, then half a step of fp16)."""
    y = x.double()
    if gamma is not None:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps) * gamma.double()
    out, size = y.clone(), y.abs()
    rd = 2 * len(inv_freq)
    for i in range(rd // 2):
        a, b = (2 * i, 2 * i + 1) if inter else (i, i + rd // 2)
        # the angle in exact rational arithmetic, reduced before it is rounded
        turns = math.fmod(float(pos) * float(inv_freq[i]), 2 * math.pi)
        cs, sn = math.cos(turns), math.sin(turns)
        out[:, a], out[:, b] = y[:, a] * cs - y[:, b] * sn, y[:, b] * cs + y[:, a] * sn
        size[:, a] = size[:, b] = torch.hypot(y[:, a], y[:, b])
    return out, 2.0 ** -11 * out.abs() + 3e-6 * size + 2.0 ** -25


def evict(c, mass, pos, nxt, keep, sink, recent):
    """kept, mass_out, pos_out rows (list per sequence and head), new lengths."""
    kept = torch.full((len(c.lens), c.k.shape[1], keep), -1, dtype=torch.int32)
    left = [min(int(n), keep) for n in c.lens]
    for s, n in enumerate(c.lens.tolist()):
        for h in range(c.k.shape[1]):
            def rank(i):
                p, m = int(pos[s, h, i]), float(mass[s, h, i])
                if p < sink or p >= int(nxt[s]) - recent:
                    return (0, 0.0, i)
                return (2, 0.0, i) if math.isnan(m) else (1, -m, i)
            best = set(sorted(range(n), key=rank)[:left[s]])
            movers = iter(sorted(i for i in best if i >= left[s]))
            for i in range(left[s]):
                kept[s, h, i] = i if i in best else next(movers)
    return kept, left
