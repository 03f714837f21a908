"""Cases of the paged key/value cache operators: what they compute, on which sizes.

Four operators, one layer's worth of decoding with a cache:

* ``rope``       a fused QKV vector per token: RMS norms of the query and key heads,
                 the rotation by position, and the keys and values written into the
                 pages of their sequences (``qk_norm_rope_append``);
* ``attention``  causal attention of each sequence's newest tokens, one or many, over
                 its cached positions (``paged_attention``);
* ``mass``       the attention weight every cached position has received, summed over
                 the new queries and the query heads that share it (``attention_mass``);
* ``evict``      the ``keep`` positions of largest mass stay, the survivors beyond
                 them move into the holes (``cache_evict``).

The cache is ``k, v`` fp16 ``[pages][kv heads][page size][head size]`` with an int32
page table ``[sequences][pages a sequence]`` and the lengths ``kv_len`` (the new
tokens included).  Tokens of all sequences lie one behind the other; sequence ``s``
has tokens ``q_start[s] .. q_start[s + 1] - 1``.
"""
import math
import random

import torch

own = False

# Rotation base and norm epsilon of the Qwen3-shaped configuration of the benchmark.
BASE, EPS = 1.0e6, 1.0e-6


def listed():
    return [
        # One token of one sequence through the 16/8-head shape: nothing but latency.
        dict(name="rope_one", op="rope", seqs=1, new_lo=1, new_hi=1, past_lo=1234, past_hi=1234, nq=16, nkv=8, hd=128, page=16, norm=True, inter=False),
        # A decode step of 61 sequences, 32/8 heads, no norms: one token each.
        dict(name="rope_batch", op="rope", seqs=61, new_lo=1, new_hi=1, past_lo=17, past_hi=4000, nq=32, nkv=8, hd=128, page=16, norm=False, inter=False),
        # Three prompts at once, 8205 tokens, with the norms.
        dict(name="rope_prompt", op="rope", seqs=3, new_lo=1000, new_hi=4500, past_lo=0, past_hi=700, nq=32, nkv=8, hd=128, page=64, norm=True, inter=False),
        # Batch-1 decoding, the 8B shape, some thousand cached positions.
        dict(name="attention_one", op="attention", seqs=1, new_lo=1, new_hi=1, past_lo=4110, past_hi=4110, nq=32, nkv=8, hd=128, page=16),
        # A decode step of 48 ragged sequences: the cache is read once, 1.6 GB of it.
        dict(name="attention_batch", op="attention", seqs=48, new_lo=1, new_hi=1, past_lo=900, past_hi=20000, nq=32, nkv=8, hd=128, page=64),
        # Four sequences checking seven drafted tokens each, heads of 64, three queries a key.
        dict(name="attention_draft", op="attention", seqs=4, new_lo=7, new_hi=7, past_lo=3001, past_hi=21000, nq=24, nkv=8, hd=64, page=32),
        # A chunk of a long prompt over what the chunks before it left in the cache.
        dict(name="attention_chunk", op="attention", seqs=1, new_lo=2048, new_hi=2048, past_lo=28711, past_hi=28711, nq=32, nkv=8, hd=128, page=16),
        # Fresh prompts of all lengths in one call, down to a single token.
        dict(name="attention_prompts", op="attention", seqs=7, new_lo=1, new_hi=4001, past_lo=0, past_hi=300, nq=16, nkv=8, hd=128, page=64),
        # The weights of one decode step, 16 sequences.
        dict(name="mass_batch", op="mass", seqs=16, new_lo=1, new_hi=1, past_lo=500, past_hi=16000, nq=32, nkv=8, hd=128, page=16),
        # The weights that a prompt's last 511 tokens give to all of it.
        dict(name="mass_chunk", op="mass", seqs=1, new_lo=511, new_hi=511, past_lo=15900, past_hi=15900, nq=32, nkv=8, hd=128, page=64),
        # A full cache of one sequence after 63 more tokens: back to its budget.
        dict(name="evict_one", op="evict", seqs=1, new_lo=1, new_hi=1, past_lo=4158, past_hi=4158, nq=32, nkv=8, hd=128, page=16, keep=4096, sink=4, recent=128),
        # Prompts of 24 sequences cut down to their budget: most of the tail goes.
        dict(name="evict_prompts", op="evict", seqs=24, new_lo=1, new_hi=1, past_lo=3000, past_hi=20000, nq=32, nkv=8, hd=128, page=64, keep=4000, sink=4, recent=256),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["rope", "attention", "attention", "attention", "mass", "evict"])
    nkv = rng.choice([1, 2, 4, 8])
    nq = nkv * rng.choice([1, 2, 3, 4, 5, 7, 8])
    c = dict(op=op, nq=nq, nkv=nkv, hd=rng.choice([64, 128]), page=rng.choice([16, 32, 64, 128]))
    if op == "rope":
        if rng.random() < 0.5:
            c.update(seqs=log(1, 200), new_lo=1, new_hi=1, past_lo=0, past_hi=log(1, 3000))
        else:
            top = log(2, 2500)
            c.update(seqs=rng.randint(1, 3), new_lo=rng.randint(1, top), new_hi=top, past_lo=0, past_hi=log(1, 2000))
        c.update(norm=rng.random() < 0.5, inter=rng.random() < 0.3)
    elif op == "evict":
        hi = log(64, 20000)
        lo = log(33, hi)
        keep = rng.randint(32, max(33, hi))
        c.update(seqs=rng.randint(1, max(1, min(24, 300000 // hi))), new_lo=1, new_hi=1, past_lo=lo, past_hi=hi, keep=keep,
                 sink=rng.randint(0, 4), recent=rng.randint(0, keep // 4))
    else:
        form = rng.choice(["one", "few", "many"])
        if form == "one":
            hi = log(2, 40000)
            c.update(seqs=rng.randint(1, max(1, min(64, 300000 // hi))), new_lo=1, new_hi=1, past_lo=rng.randint(1, hi), past_hi=hi)
        elif form == "few":
            hi = log(2, 20000)
            top = rng.randint(2, 40)
            c.update(seqs=rng.randint(1, 8), new_lo=rng.randint(1, top), new_hi=top, past_lo=0, past_hi=hi)
        else:
            top = log(41, 1500)
            c.update(seqs=rng.randint(1, 3), new_lo=rng.randint(1, top), new_hi=top, past_lo=0, past_hi=log(1, 10000))
    return c


# ------------------------------------------------------------------ sizes


def _spread(lo, hi, n, salt):
    """n lengths between lo and hi, even in their logarithm, in a fixed mixed order."""
    if n == 1:
        return [hi]
    a, b = math.log(lo + 1), math.log(hi + 1)
    v = [int(round(math.exp(a + (b - a) * i / (n - 1)))) - 1 for i in range(n)]
    random.Random(salt * 1000 + n).shuffle(v)
    return v


def _lengths(case):
    """New tokens and cached positions (the new ones included) of each sequence."""
    new = _spread(case["new_lo"], case["new_hi"], case["seqs"], 1)
    past = _spread(case["past_lo"], case["past_hi"], case["seqs"], 2)
    return new, [a + b for a, b in zip(new, past)]


def _pairs(case):
    """(query, key) pairs that the causal mask leaves, over one query head."""
    return sum(n * (t - n) + n * (n + 1) // 2 for n, t in zip(*_lengths(case)))


def work(case):
    new, lens = _lengths(case)
    nq, nkv, hd, toks, kv = case["nq"], case["nkv"], case["hd"], sum(new), sum(lens)
    if case["op"] == "rope":
        heads = nq + 2 * nkv
        return {"bytes": toks * (heads * hd * 4 + 8 * nkv + 4), "flops": toks * (nq + nkv) * hd * (7 if case["norm"] else 3)}
    if case["op"] == "attention":
        return {"bytes": kv * nkv * hd * 4 + toks * nq * (hd * 4 + 4), "flops": 4 * hd * nq * _pairs(case)}
    if case["op"] == "mass":
        return {"bytes": kv * nkv * (hd * 2 + 8) + toks * nq * (hd * 2 + 4), "flops": 2 * hd * nq * _pairs(case)}
    kept = [min(t, case["keep"]) for t in lens]
    moved = sum((t - k) * k // t for t, k in zip(lens, kept))  # the tail's share of the survivors
    return {"bytes": nkv * (8 * kv + 12 * sum(kept) + moved * hd * 8), "flops": 8 * nkv * kv}


# ----------------------------------------------------------------- inputs


def prepare(case, seed):
    new, lens = _lengths(case)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dev, S, nq, nkv, hd, ps = "cuda", case["seqs"], case["nq"], case["nkv"], case["hd"], case["page"]
    toks = sum(new)

    def normal(*shape, scale=1.0):
        return (torch.randn(shape, generator=g, device=dev) * scale).half()

    # Pages are handed out in mixed order from a pool with a few to spare.
    need = [(t + ps - 1) // ps for t in lens]
    per = max(need) + 1
    order = torch.randperm(sum(need) + 5, generator=g, device=dev).int()
    table = torch.zeros(S, per, dtype=torch.int32, device=dev)
    at = 0
    for s, n in enumerate(need):
        table[s, :n] = order[at:at + n]
        at += n
    pool = (sum(need) + 5, nkv, ps, hd)
    st = dict(case=case, op=case["op"], lens=lens, new=new, longest=max(lens), most=max(new), table=table,
              k=normal(*pool), v=normal(*pool),
              kv_len=torch.tensor(lens, dtype=torch.int32, device=dev),
              q_start=torch.tensor([0] + [sum(new[:i + 1]) for i in range(S)], dtype=torch.int32, device=dev))
    cap = per * ps
    if case["op"] == "rope":
        shift = torch.randint(0, 120000, (S,), generator=g, device=dev)  # positions evicted before
        seq = torch.repeat_interleave(torch.arange(S, device=dev), torch.tensor(new, device=dev))
        j = torch.arange(toks, device=dev) - st["q_start"][seq]
        st.update(qkv=normal(toks, (nq + 2 * nkv) * hd, scale=1.5),
                  positions=(shift[seq] + st["kv_len"][seq] - torch.tensor(new, device=dev)[seq] + j).int(),
                  inv_freq=(BASE ** (-torch.arange(0, hd, 2, dtype=torch.float64) / hd)).float().to(dev),
                  q_norm=(1 + normal(hd, scale=0.05)) if case["norm"] else None,
                  k_norm=(1 + normal(hd, scale=0.05)) if case["norm"] else None,
                  q_out=torch.zeros(toks, nq * hd, dtype=torch.float16, device=dev),
                  entry_pos=torch.zeros(S, nkv, cap, dtype=torch.int32, device=dev),
                  entry_mass=torch.ones(S, nkv, cap, device=dev))
    elif case["op"] in ("attention", "mass"):
        st["q"] = normal(toks, nq * hd, scale=2.0)
        if case["op"] == "mass":
            st.update(mass=torch.rand(S, nkv, cap, generator=g, device=dev), mass_out=torch.zeros(S, nkv, cap, device=dev))
            score, _ = _scores(st)
            st["lse"] = _tokens(st, torch.logsumexp(score, -1, keepdim=True)).view(toks, nq).contiguous()
            del score
    else:
        mass = torch.exp(2 * torch.randn(S, nkv, cap, generator=g, device=dev))
        mass[torch.rand(S, nkv, cap, generator=g, device=dev) < 0.1] = 0.0  # never looked at: many ties
        # positions: distinct, with gaps, roughly rising (holes were filled before)
        pos = torch.cumsum(torch.randint(1, 3, (S, nkv, cap), generator=g, device=dev), -1)
        mixed = torch.argsort(torch.rand(S, nkv, cap, generator=g, device=dev) + torch.arange(cap, device=dev) * (4.0 / cap), -1)
        inside = torch.arange(cap, device=dev) < st["kv_len"][:, None, None]
        pos = torch.gather(pos, -1, torch.argsort(torch.argsort(torch.where(inside, mixed, cap + mixed), -1), -1))
        st.update(mass=mass, entry_pos=pos.int(),
                  next_pos=(torch.where(inside, pos, -1).amax((1, 2)) + 1).int(),
                  mass_out=torch.zeros(S, nkv, cap, device=dev), pos_out=torch.zeros(S, nkv, cap, dtype=torch.int32, device=dev),
                  kept=torch.zeros(S, nkv, case["keep"], dtype=torch.int32, device=dev),
                  kv_len_out=torch.zeros(S, dtype=torch.int32, device=dev))
    if own:  # the handle of the cache, which a program makes once
        import bit_group_quantized_qgemv_gb300 as q
        st["cache"] = q.kv_cache(st["k"], st["v"], st["table"], st["kv_len"])
    return st


# ------------------------------------------------------------- plain form


def _rows(st):
    """Sequence and place within it of every new token."""
    toks = torch.arange(sum(st["new"]), device="cuda")
    seq = torch.searchsorted(st["q_start"][1:].contiguous(), toks.int(), right=True)
    return seq, toks - st["q_start"][seq]


def _gather(st, pool):
    """The cached rows of all sequences, fp32 [sequence][kv head][position][head size]."""
    ps = st["case"]["page"]
    i = torch.arange(st["longest"], device="cuda")
    return pool[st["table"][:, i // ps].long(), :, i % ps].permute(0, 2, 1, 3).float()


def _scores(st):
    """Masked scores [sequence][kv head][token x query head of the group][position], and the mask."""
    c = st["case"]
    S, nq, nkv, hd, n = c["seqs"], c["nq"], c["nkv"], c["hd"], st["most"]
    seq, j = _rows(st)
    q = torch.zeros(S, n, nq, hd, device="cuda")
    q[seq, j] = st["q"].view(-1, nq, hd).float()
    q = q.view(S, n, nkv, nq // nkv, hd).permute(0, 2, 1, 3, 4).reshape(S, nkv, -1, hd)
    score = torch.matmul(q, _gather(st, st["k"]).transpose(-1, -2)).mul_(hd ** -0.5)
    new = st["q_start"][1:] - st["q_start"][:-1]
    row = torch.arange(n, device="cuda").repeat_interleave(nq // nkv)
    last = (st["kv_len"] - new)[:, None] + row
    hidden = torch.arange(st["longest"], device="cuda") > last[:, None, :, None]
    hidden = hidden | (row >= new[:, None])[:, None, :, None]
    return score.masked_fill_(hidden, -math.inf), hidden


def _tokens(st, rows):
    """[sequence][kv head][token x group][any] back to [token][query head][any]."""
    c = st["case"]
    seq, j = _rows(st)
    x = rows.view(c["seqs"], c["nkv"], st["most"], c["nq"] // c["nkv"], -1).permute(0, 2, 1, 3, 4)
    return x[seq, j].reshape(len(seq), c["nq"], -1)


def _plain_rope(st):
    c = st["case"]
    nq, nkv, hd = c["nq"], c["nkv"], c["hd"]
    x = st["qkv"].view(-1, nq + 2 * nkv, hd)
    qk, v = x[:, :nq + nkv].float(), x[:, nq + nkv:]
    if c["norm"]:
        gamma = torch.cat([st["q_norm"].float().expand(nq, hd), st["k_norm"].float().expand(nkv, hd)])
        qk = qk * torch.rsqrt(qk.square().mean(-1, keepdim=True) + EPS) * gamma
    angle = st["positions"].double()[:, None, None] * st["inv_freq"].double()
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    a, b = (qk[..., 0::2], qk[..., 1::2]) if c["inter"] else (qk[..., :hd // 2], qk[..., hd // 2:])
    a, b = a * cos - b * sin, b * cos + a * sin
    qk = (torch.stack([a, b], -1).flatten(-2) if c["inter"] else torch.cat([a, b], -1)).half()
    seq, j = _rows(st)
    new = st["q_start"][1:] - st["q_start"][:-1]
    at = (st["kv_len"] - new)[seq] + j
    page, off = st["table"][seq, at // c["page"]].long(), at % c["page"]
    st["k"][page, :, off] = qk[:, nq:]
    st["v"][page, :, off] = v
    st["entry_pos"][seq, :, at] = st["positions"][:, None].expand(-1, nkv)
    st["entry_mass"][seq, :, at] = 0.0
    st["q_out"].copy_(qk[:, :nq].reshape(st["q_out"].shape))
    return [st["q_out"], st["k"], st["v"], st["entry_pos"], st["entry_mass"]]


def _plain_attention(st):
    c = st["case"]
    score, _ = _scores(st)
    m = score.amax(-1, keepdim=True)
    p = torch.exp(score.sub_(torch.where(torch.isinf(m), 0.0, m)))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, _gather(st, st["v"])) / torch.where(total > 0, total, 1.0)
    return [_tokens(st, o).half().view(-1, c["nq"] * c["hd"]), _tokens(st, m + torch.log(total)).view(-1, c["nq"])]


def _plain_mass(st):
    c = st["case"]
    score, hidden = _scores(st)
    seq, j = _rows(st)
    lse = torch.zeros(c["seqs"], st["most"], c["nq"], device="cuda")
    lse[seq, j] = st["lse"]
    lse = lse.view(c["seqs"], st["most"], c["nkv"], -1).permute(0, 2, 1, 3).reshape(c["seqs"], c["nkv"], -1, 1)
    got = torch.exp(score - lse).masked_fill_(hidden, 0.0).sum(2)
    inside = torch.arange(st["longest"], device="cuda") < st["kv_len"][:, None, None]
    out = st["mass_out"][:, :, :st["longest"]]
    out.copy_(torch.where(inside, st["mass"][:, :, :st["longest"]] + got, out))
    return [st["mass_out"]]


def _plain_evict(st):
    c = st["case"]
    cap, keep, n = st["mass"].shape[-1], c["keep"], st["kv_len"][:, None, None]
    i = torch.arange(cap, device="cuda").expand_as(st["mass"])
    inside, pos = i < n, st["entry_pos"]
    safe = (pos < c["sink"]) | (pos >= (st["next_pos"] - c["recent"])[:, None, None])
    rank = torch.where(inside, torch.where(safe, math.inf, st["mass"]), -1.0)
    order = torch.sort(rank, dim=-1, descending=True, stable=True).indices
    left = torch.clamp(n, max=keep)
    stays = torch.zeros_like(inside).scatter_(-1, order, i < left)
    hole, mover = ~stays & (i < left), stays & (i >= left)
    # the k-th hole takes the k-th mover
    hole_at = torch.argsort((~hole).byte(), dim=-1, stable=True)
    mover_at = torch.argsort((~mover).byte(), dim=-1, stable=True)
    source = torch.where(i < left, i, -1).scatter_(-1, hole_at, torch.where(i < hole.sum(-1, keepdim=True), mover_at, torch.where(hole_at < left, hole_at, -1)))
    take = torch.clamp(source, min=0)
    st["mass_out"].copy_(torch.where(i < left, torch.gather(st["mass"], -1, take), st["mass_out"]))
    st["pos_out"].copy_(torch.where(i < left, torch.gather(pos, -1, take), st["pos_out"]))
    st["kept"].fill_(-1)
    st["kept"][:, :, :min(keep, cap)] = source[:, :, :keep].int()
    st["kv_len_out"].copy_(left.view(-1))
    s, h, to = torch.nonzero((source != i) & (source >= 0), as_tuple=True)
    frm, ps = source[s, h, to], c["page"]
    a, b = st["table"][s, frm // ps].long(), st["table"][s, to // ps].long()
    st["k"][b, h, to % ps] = st["k"][a, h, frm % ps]
    st["v"][b, h, to % ps] = st["v"][a, h, frm % ps]
    return [st["kept"], st["mass_out"], st["pos_out"], st["kv_len_out"], st["k"], st["v"]]


def run(st):
    if not own:
        return {"rope": _plain_rope, "attention": _plain_attention, "mass": _plain_mass, "evict": _plain_evict}[st["op"]](st)
    import bit_group_quantized_qgemv_gb300 as q
    c, cache = st["case"], st["cache"]
    if st["op"] == "rope":
        q.qk_norm_rope_append(cache, st["qkv"], st["q_start"], st["positions"], st["inv_freq"], interleaved=c["inter"],
                              q_norm=st["q_norm"], k_norm=st["k_norm"], eps=EPS, q_out=st["q_out"],
                              entry_pos=st["entry_pos"], entry_mass=st["entry_mass"])
        return [st["q_out"], st["k"], st["v"], st["entry_pos"], st["entry_mass"]]
    if st["op"] == "attention":
        return list(q.paged_attention(cache, st["q"], st["q_start"], max_q=st["most"], want_lse=True))
    if st["op"] == "mass":
        return [q.attention_mass(cache, st["q"], st["q_start"], st["lse"], max_q=st["most"], mass=st["mass"], mass_out=st["mass_out"])]
    q.cache_evict(cache, st["mass"], st["entry_pos"], st["next_pos"], c["keep"], n_sink=c["sink"], n_recent=c["recent"],
                  kept=st["kept"], mass_out=st["mass_out"], pos_out=st["pos_out"], kv_len_out=st["kv_len_out"])
    return [st["kept"], st["mass_out"], st["pos_out"], st["kv_len_out"], st["k"], st["v"]]


# ---------------------------------------------------- definition, 64 bits


def _sequence(st, s, pool):
    """Sequence s's cached rows, 64 bits [position][kv head][head size]."""
    n, ps = st["lens"][s], st["case"]["page"]
    pages = pool.index_select(0, st["table"][s, :(n + ps - 1) // ps].long())
    return pages.transpose(1, 2).reshape(-1, pool.shape[1], pool.shape[3])[:n].double()


def exact(case, seed):
    st = prepare(case, seed)
    nq, nkv, hd, ps, S = case["nq"], case["nkv"], case["hd"], case["page"], case["seqs"]
    grp, first = nq // nkv, [0]
    for n in st["new"]:
        first.append(first[-1] + n)
    if case["op"] == "rope":
        x = st["qkv"].double().view(-1, nq + 2 * nkv, hd)
        out = [x[:, :nq], x[:, nq:nq + nkv], x[:, nq + nkv:]]
        ang = st["positions"].double()[:, None] * st["inv_freq"].double()[None]
        turn = torch.polar(torch.ones_like(ang), ang)[:, None]
        for w, gamma in ((0, st["q_norm"]), (1, st["k_norm"])):
            y = out[w]
            if gamma is not None:
                y = y / torch.sqrt((y * y).sum(-1, keepdim=True) / hd + EPS) * gamma.double()
            z = torch.view_as_complex((y.reshape(*y.shape[:2], hd // 2, 2) if case["inter"]
                                       else torch.stack(y.chunk(2, -1), -1)).contiguous()) * turn
            z = torch.view_as_real(z)
            out[w] = z.flatten(-2) if case["inter"] else torch.cat([z[..., 0], z[..., 1]], -1)
        kc, vc, pos, mass = st["k"].double(), st["v"].double(), st["entry_pos"], st["entry_mass"].double()
        for s in range(S):
            a, b, t = first[s], first[s + 1], st["lens"][s]
            i = torch.arange(t - (b - a), t, device="cuda")
            pg = st["table"][s, i // ps].long()
            kc[pg, :, i % ps], vc[pg, :, i % ps] = out[1][a:b], out[2][a:b]
            pos[s, :, t - (b - a):t] = st["positions"][a:b]
            mass[s, :, t - (b - a):t] = 0
        return [out[0].reshape(-1, nq * hd), kc, vc, pos, mass]
    if case["op"] in ("attention", "mass"):
        q = st["q"].double().view(-1, nkv, grp, hd)
        o = torch.zeros(len(q), nkv, grp, hd, dtype=torch.float64, device="cuda")
        lse = torch.zeros(len(q), nkv, grp, dtype=torch.float64, device="cuda")
        mass = st["mass_out"].double() if case["op"] == "mass" else None
        for s in range(S):
            a, b, t = first[s], first[s + 1], st["lens"][s]
            if a == b:
                continue
            K, V = _sequence(st, s, st["k"]), _sequence(st, s, st["v"])
            seen = torch.arange(t, device="cuda")[None] <= torch.arange(t - (b - a), t, device="cuda")[:, None]
            for h in range(nkv):
                z = torch.einsum("igd,jd->igj", q[a:b, h], K[:, h]) / math.sqrt(hd)
                if mass is not None:
                    w = torch.exp(z - st["lse"].double().view(-1, nkv, grp)[a:b, h, :, None]) * seen[:, None]
                    mass[s, h, :t] = st["mass"][s, h, :t].double() + w.sum((0, 1))
                    continue
                z = torch.where(seen[:, None], z, -math.inf)
                lse[a:b, h] = torch.logsumexp(z, -1)
                o[a:b, h] = torch.einsum("igj,jd->igd", torch.softmax(z, -1), V[:, h])
        return [mass] if mass is not None else [o.reshape(-1, nq * hd), lse.reshape(-1, nq)]
    # evict: sets and copies in numpy, head by head
    import numpy as np
    mass, pos, nxt = (st[k].cpu().numpy() for k in ("mass", "entry_pos", "next_pos"))
    kept, m2, p2 = (st[k].cpu().numpy() for k in ("kept", "mass_out", "pos_out"))
    left, kept[:] = [min(t, case["keep"]) for t in st["lens"]], -1
    k, v = st["k"], st["v"]
    for s in range(S):
        for h in range(nkv):
            t, n = st["lens"][s], left[s]
            safe = (pos[s, h, :t] < case["sink"]) | (pos[s, h, :t] >= nxt[s] - case["recent"])
            best = np.lexsort((np.arange(t), -mass[s, h, :t].astype(np.float64), ~safe))[:n]
            src = np.arange(n)
            src[np.setdiff1d(src, best)] = np.sort(best[best >= n])
            kept[s, h, :n], m2[s, h, :n], p2[s, h, :n] = src, mass[s, h, src], pos[s, h, src]
            to = np.flatnonzero(src != np.arange(n))
            to, frm = torch.from_numpy(to).cuda(), torch.from_numpy(src[to]).cuda()
            pa, pb = st["table"][s, frm // ps].long(), st["table"][s, to // ps].long()
            k[pb, h, to % ps], v[pb, h, to % ps] = k[pa, h, frm % ps], v[pa, h, frm % ps]
    return [torch.from_numpy(kept), torch.from_numpy(m2).double(), torch.from_numpy(p2), torch.tensor(left, dtype=torch.int32), k.double(), v.double()]
