"""The many-rows attention kernel's sharing out of its work, run on the CPU (a warp of
32 contexts, units_on_cpu.cpp): whatever the sequences, every tile of every unit goes out
exactly once, and the parts of a cut unit lie where their join looks for them."""
import os
import subprocess

import numpy as np
import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "bit_group_quantized_qgemv_gb300", "csrc")
TILE, UNIT = 128, 256


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("units") / "units")
    subprocess.run(["g++", "-O2", "-std=c++17", "-I", CSRC, "-w", os.path.join(HERE, "units_on_cpu.cpp"),
                    "-o", exe], check=True)
    return exe


def share_out(program, seqs, n_kv, group, cut, blocks=152, max_q=None):
    """Segments (block, s, h, r0, rows, off, j0, j1, slot) and cut units (block, parts, s, h, r0)."""
    max_q = max_q or max(m for m, _ in seqs)
    text = " ".join(str(v) for v in [blocks, n_kv, group, max_q, int(cut), len(seqs)] +
                    [v for pair in seqs for v in pair])
    r = subprocess.run([program], input=text, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.endswith("end\n"), r.stdout[-300:]
    lines = [ln.split() for ln in r.stdout.splitlines()[:-1]]
    return ([tuple(map(int, ln[1:])) for ln in lines if ln[0] == "g"],
            {int(ln[1]): tuple(map(int, ln[2:])) for ln in lines if ln[0] == "u"})


def check(program, seqs, n_kv, group, cut, **kw):
    segs, cuts = share_out(program, seqs, n_kv, group, cut, **kw)
    max_q = kw.get("max_q") or max(m for m, _ in seqs)
    want = {}                                     # unit -> its tiles
    for s, (m, n) in enumerate(seqs):
        rows = min(m, max_q) * group
        for r0 in range(0, rows, UNIT):
            see = min(n, n - m + (min(rows, r0 + UNIT) - 1) // group + 1)
            for h in range(n_kv):
                want[s, h, r0] = max(1, -(-see // TILE))
    got = {u: [] for u in want}
    for b, s, h, r0, rows, off, j0, j1, slot in segs:
        m, n = seqs[s]
        assert (rows, off) == (min(m, max_q) * group, n - m)
        got[s, h, r0].append((j0, j1, b, slot))
    n_cut = 0
    for u, t in want.items():
        parts = sorted(got[u])
        assert parts and parts[0][0] == 0 and parts[-1][1] == t, (u, t, parts)
        for (_, e, *_), (j, *_) in zip(parts, parts[1:]):
            assert e == j, (u, t, parts)
        if len(parts) == 1:
            assert parts[0][3] == -1
            continue
        n_cut += 1
        first = parts[0][2]
        assert cuts[first] == (len(parts), *u)
        for p, (j0, _, b, slot) in enumerate(parts):
            assert b == first + p and slot == 2 * b + (p == 0)
    assert n_cut == len(cuts)
    return n_cut


@pytest.mark.parametrize("seed", range(24))
@pytest.mark.parametrize("cut", [False, True])
def test_every_tile_once(program, seed, cut):
    g = np.random.default_rng(seed)
    n_seqs = int(g.choice([1, 2, 3, 7, 16, 17, 32, 33, 50]))
    longest = int(g.choice([20, 300, 3000]))
    seqs = [(int(m), int(max(0, m + g.integers(-10, longest)))) for m in g.integers(0, longest, n_seqs)]
    seqs[0] = (longest, longest + 5)
    check(program, seqs, int(g.choice([1, 2, 8])), int(g.choice([1, 3, 4, 7, 8])), cut,
          blocks=int(g.choice([13, 148, 152, 160])))


def test_cut_and_whole(program):
    """The rule's examples: 2048 tokens over 30759 entries and 64 over 8064 are cut, 1200 over 9400 not."""
    assert check(program, [(2048, 30759)], 8, 4, True) > 0
    assert check(program, [(64, 8064)], 8, 4, True) > 0
    assert check(program, [(1200, 9400)], 8, 4, True) == 0


def test_more_tokens_than_declared(program):
    check(program, [(700, 900), (20, 20)], 2, 4, True, max_q=300)


# Spans (tiles and kUnitCost) past 2^31: of one head, 513 units of 2^22 tiles (131,328 rows
# over 2^29 entries) alone and among short sequences; of the heads of one row tile, 1024 x
# 2^22 (a page table may repeat its pages, so the cache need not be that large).
LONG = [([(131328, 1 << 29)], 1, 1), ([(5, 9), (131328, 1 << 29), (0, 4)], 2, 1),
        ([(16500, 1 << 29)], 1, 8), ([(16500, 1 << 29)] * 3, 3, 8), ([(256, 1 << 29)], 1024, 1)]


@pytest.mark.parametrize("cut", [False, True])
@pytest.mark.parametrize("case", range(len(LONG)))
def test_more_than_2_31_tiles(program, case, cut):
    seqs, n_kv, group = LONG[case]
    n_cut = check(program, seqs, n_kv, group, cut)
    assert n_cut > 0 if cut else n_cut == 0
