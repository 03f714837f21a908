"""What the blocks of a cluster tell one another in the kernels of the MXFP4 products
(csrc/mx_product.cu, csrc/mx_pair.cu), without a GPU."""
import os
import random
import re
import subprocess

import pytest

import bit_group_quantized_qgemv_gb300 as q
from mx_cluster_shapes import ALONE, PAIRS_ODD, ROWS_ODD, SHARED
from test_mx_plan import CLUSTERS, plans, program  # noqa: F401
from test_mx_protocol import Barrier, play, wait

CSRC = os.path.join(os.path.dirname(q.__file__), "csrc")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


# ------------------------------------------------------------------- scopes

@pytest.mark.parametrize("name,shared", [("mx_pair.cu", ("full", "empty", "acc_full", "acc_empty")),
                                         ("mx_product.cu", ("part_full", "part_done"))])
def test_waits_for_other_blocks_are_in_the_clusters_scope(name, shared):
    """Memory is ordered between two blocks by an arrival and a wait that both have the cluster's
    scope; what an arrival or a wait without one (the block's own) orders is undefined there."""
    waits = re.findall(r"step_wait(<true>)?\(smem_u32\(&bars\.(\w+)", source(name))
    assert {bar for _, bar in waits} >= set(shared)
    for scope, bar in waits:
        assert (scope == "<true>") == (bar in shared), f"{name}: {bar}"


def test_arrivals_at_other_blocks_are_in_the_clusters_scope():
    names = [n for n in sorted(os.listdir(CSRC)) if n.endswith((".cu", ".cuh"))]
    found = 0
    for name in names:
        text = source(name)
        for arrive in re.findall(r"mbarrier\.arrive[\w.:]*shared::cluster[\w.:]*", text):
            found += 1
            assert ".cluster.shared::cluster" in arrive, f"{name}: {arrive}"
            if ".relaxed." in arrive:                   # (a fence before it, in the same function)
                body = text[:text.index(arrive)].rsplit("__device__", 1)[1]
                assert "fence.release.sync_restrict::shared::cta.cluster" in body, f"{name}: {arrive}"
    assert found > 0
    wait = source("qgemv_device.cuh").split("bool mbar_try_wait_cluster", 1)[1].split("\n}\n", 1)[0]
    assert "relaxed.cluster.shared::cta" in wait
    loop = source("kv_cache.cuh").split("void step_wait(", 1)[1].split("\n}\n", 1)[0]
    assert loop.index("mbar_try_wait_cluster") < loop.index("if (CLUSTER) mbar_acquire_cluster()") < loop.index("__syncwarp")


# ----------------------------------------------------- how many run at a time

def test_numbers_of_clusters(tmp_path):
    exe = str(tmp_path / "clusters")
    here = os.path.dirname(os.path.abspath(__file__))
    subprocess.run(["g++", "-O2", "-std=c++17", "-I", CSRC, os.path.join(here, "clusters_on_cpu.cpp"), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and r.stdout == "done\n", r.stderr


def test_each_kernel_is_asked():
    """A table for each kernel (a template of the kernel, not of its type, which they share)."""
    assert re.search(r"template <auto\* kKernel>\s+int clusters_at_a_time\(", source("mx_product.cuh"))
    pair = source("mx_pair.cu")
    for kernel in ("true, true", "true, false", "false, true", "false, false"):
        assert f"clusters_at_a_time<mx_pair_kernel<{kernel}>>" in pair
    assert "clusters_at_a_time<k>" in source("mx_product.cu")


# ------------------------------------------------------- sums that are shared

def share(rng, split, tokens, counts, halves=(0, 1), quarters=2, wait_done=True, behind=True):
    """The results of a cluster's blocks (csrc/mx_product.cu): each rank's sums of every column go to
    the rank that finishes it, m % split, tile after tile of counts columns.  A place is written
    when its message arrives, which is any time and in any order after it was sent."""
    out = len(halves) * quarters
    full, done = [Barrier(1) for _ in range(split)], [Barrier(out * split) for _ in range(split)]
    held = [{} for _ in range(split)]                      # place: the tile whose sum is there
    later = []

    def arrive(rank, place, tile):
        def f():
            assert place not in held[rank], "a sum is written over before it was read"
            held[rank][place] = tile
            full[rank].complete()
        return f

    def results(rank, half, quarter):
        for n, count in enumerate(counts):
            own = (count - rank + split - 1) // split
            for step in ("done", "expect") if behind else ("expect", "done"):
                if step == "expect" and half == 0 and quarter == 0:
                    full[rank].arrive(tx=max(own, 0) * split * quarters)
                    yield
                if step == "done" and n > 0 and wait_done:
                    yield from wait(done[rank], (n - 1) & 1, n)
            for m in [m for m in range(count) if (m // 4) % len(halves) == half]:
                later.insert(rng.randint(0, len(later)), arrive(m % split, (rank, m // split, quarter), n))
                if rng.random() < 0.3:
                    yield
            yield from wait(full[rank], n & 1, n + 1)
            for j in range(half, own, len(halves)):
                for sender in range(split):
                    assert held[rank].pop((sender, j, quarter)) == n
                yield
            if n + 1 < len(counts):
                for to in range(split):
                    done[to].arrive()
                    yield

    play(rng, [results(r, h, k) for r in range(split) for h in halves for k in range(quarters)], later)
    assert not any(held)
    for b in full + done:
        assert b.pending == b.count and b.tx == 0


def some_sums(rng):
    tokens = rng.randint(1, 20)
    return dict(split=rng.choice([2, 4, 8]), tokens=tokens,
                counts=[tokens if rng.random() < 0.7 else rng.randint(1, tokens) for _ in range(rng.randint(1, 6))])


@pytest.mark.parametrize("seed", range(4))
def test_shared_sums(seed):
    rng = random.Random(seed)
    for _ in range(12):
        share(rng, **some_sums(rng))


@pytest.mark.parametrize("wrong", ["wait_done", "behind"])
def test_the_schedules_find_what_is_wrong_in_sharing(wrong):
    """Without the wait for the readers some schedule writes over a sum that has not been read.  Where the
    bytes of a tile are expected before that wait, a rank that finishes no column (there are fewer than
    ranks) ends a phase that its other warps have not seen end the phase before, and they wait forever."""
    rng = random.Random(1)
    with pytest.raises(AssertionError, match="no warp gets any further" if wrong == "behind" else None):
        for _ in range(100):
            share(rng, **some_sums(rng), **{wrong: False})


def test_order_of_the_kernel_in_sharing():
    body = source("mx_product.cu")
    assert body.count("mbar_arrive_expect_tx(smem_u32(&bars.part_full)") == 1
    assert body.index("step_wait<true>(smem_u32(&bars.part_done)") < body.index("mbar_arrive_expect_tx(smem_u32(&bars.part_full)")


# ------------------------------------------------------------- fp16 rows

def test_every_use_of_fp16_rows_is_behind_a_wait_for_them():
    """Two warps take every other step, counted over all tiles; the columns of a step are waited for in some
    of the tiles, and each warp has to have waited for those of every step that it uses."""
    when = re.findall(r"if \(SPLIT && ([^)]*)\) step_wait\(smem_u32\(&bars\.rows\[k - k0\]\)", source("mx_product.cu"))
    assert len(when) == 1
    for steps in range(1, 12):
        seen, odd = set(), 0
        for n in range(6):
            for k in range(steps):
                if eval(when[0], {"n": n}):
                    seen.add((odd, k))
                assert (odd, k) in seen, f"{steps} steps: step {k} of tile {n}"
                odd ^= 1


# --------------------------------------------------------- sizes of the tests

def test_sizes_reach_several_tiles_of_a_cluster(program):  # noqa: F811
    at_a_time = dict(zip((1, 2, 4, 8), CLUSTERS))
    for (split, shape), p in zip(SHARED, plans(program, [s for _, s in SHARED])):
        assert p["split"] == split and not p["faster"], shape
        assert p["row_tiles"] * p["tok_tiles"] > 2 * at_a_time[split], shape
    assert {(s, shape[3], shape[4]) for s, shape in SHARED} >= {(2, 0, 1), (4, 0, 1), (8, 0, 1), (4, 0, 0), (8, 0, 0), (4, 1, 0)}
    rounds = set()
    for shape, p in zip(PAIRS_ODD, plans(program, PAIRS_ODD)):
        steps = shape[2] // 128
        assert p["faster"] and p["two2"] and steps % 2 == 1 and steps >= 3, shape
        rounds.add((shape[3], min(3, -(-p["row_tiles2"] * p["tok_tiles2"] // CLUSTERS[1]))))
    assert {(0, 2), (0, 3), (1, 3)} <= rounds
    for shape, p in zip(ALONE, plans(program, ALONE)):
        assert p["split"] == 1 and not p["faster"] and p["row_tiles"] * p["tok_tiles"] > CLUSTERS[0], shape
    for shape, p in zip(ROWS_ODD, plans(program, ROWS_ODD)):
        assert p["split"] == 1 and -(-shape[2] // 128) % 2 == 1 and p["row_tiles"] > CLUSTERS[0], shape
