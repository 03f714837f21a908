"""How products with MXFP4 weights are cut into tiles (csrc/mx_plan.h), on the CPU: every plan
fits a multiprocessor and covers the product, for every size that the library takes."""
import os
import random
import subprocess

import pytest

import mx_reference as ref

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "bit_group_quantized_qgemv_gb300", "csrc")
CLUSTERS = (152, 76, 36, 15)
NAMES = "ok cols tokens split stages row_tiles tok_tiles row_steps pair rows_first smem " \
        "by_two faster cols2 stages2 row_tiles2 tok_tiles2 smem2 two2".split()


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("plans") / "plans")
    subprocess.run(["g++", "-O2", "-std=c++17", "-I", CSRC, os.path.join(HERE, "plans_on_cpu.cpp"), "-o", exe], check=True)
    return exe


def plans(program, shapes, clusters=CLUSTERS):
    text = "".join(" ".join(str(int(v)) for v in (*s, *clusters)) + "\n" for s in shapes)
    r = subprocess.run([program], input=text, capture_output=True, text=True, check=True, timeout=300)
    return [dict(zip(NAMES, map(int, ln.split()))) for ln in r.stdout.splitlines()]


def check(shape, p, two=True):
    M, N, K, gated, fp16 = shape
    w, steps = 2 if gated else 1, -(-K // 128)
    assert p["ok"], shape
    assert p["cols"] % 16 == 0 and 16 <= p["cols"] <= 240
    assert p["stages"] >= 4 and p["stages"] % 2 == 0 and p["stages"] <= 16
    assert p["split"] in (1, 2, 4, 8) and p["split"] <= steps          # every rank has a step
    assert p["row_tiles"] * 128 >= N and p["tok_tiles"] * p["tokens"] >= M
    assert (p["tok_tiles"] - 1) * p["tokens"] < M                       # no tile without rows
    accumulators = 2 * (2 if gated or p["pair"] else 1) * p["cols"]
    assert accumulators + 32 <= 512
    stage = w * 16384 + (0 if fp16 else p["cols"] * 128) + 512 * (w + (0 if fp16 else 1 + (p["cols"] > 128)))
    rows = p["row_steps"] * (p["cols"] * 128 + 512)
    part = w * -(-p["tokens"] // p["split"]) * p["split"] * 512 if p["split"] > 1 else 0
    out = 16384 if not fp16 and not gated and p["split"] == 1 else 0
    assert p["smem"] >= 1024 + p["stages"] * stage + rows + part + out
    assert p["smem"] + 1024 <= 227 * 1024                              # and what is static
    assert p["by_two"] == (not fp16 and K % 128 == 0 and two)
    if p["by_two"]:                                                     # two blocks that share their tiles
        assert p["cols2"] % 32 == 0 and (4 if p["two2"] else 2) * p["cols2"] + 32 <= 512
        assert p["stages2"] >= 4 and p["stages2"] % 2 == 0 and p["stages2"] <= 16
        assert p["row_tiles2"] * (128 if gated else 256) >= N and p["tok_tiles2"] * p["cols2"] >= M
        assert (p["tok_tiles2"] - 1) * p["cols2"] < M
        stage = 16384 + p["cols2"] * 64 + 512 * (3 if p["cols2"] > 128 else 2)
        assert p["smem2"] >= 1024 + p["stages2"] * stage + 16384 and p["smem2"] + 1024 <= 227 * 1024
        assert p["smem2"] > 114 * 1024                                  # one block a multiprocessor
    if fp16:
        assert p["tok_tiles"] == 1 and p["tokens"] == M and 3 * M <= p["cols"] <= 32
        assert p["pair"] and p["row_steps"] * p["split"] >= steps and p["row_steps"] <= 64


@pytest.mark.parametrize("clusters", [CLUSTERS, (152, 76, 38, 19), (148, 74, 0, 0), (152, 0, 0, 0)])
def test_random_sizes(program, clusters):
    rng = random.Random(1)
    shapes = []
    for _ in range(3000):
        K = 32 * int(2 ** rng.uniform(0, 11))
        N, M = int(2 ** rng.uniform(0, 18)), int(2 ** rng.uniform(0, 17))
        shapes.append((M, N, K, rng.random() < 0.4, 0))
    for s, p in zip(shapes, plans(program, shapes, clusters)):
        check(s, p, clusters[1] > 0)


def test_fp16_rows_of_every_length(program):
    shapes = [(M, N, K, 0, 1) for M in range(1, 9) for N in (1, 4096, 151936) for K in range(32, 28673, 32 * 7)] + \
             [(M, 4096, 28672, 0, 1) for M in range(1, 9)]
    got = plans(program, shapes)
    for s, p in zip(shapes, got):
        check(s, p)
    by = {}
    for (M, N, K, _, _), p in zip(shapes, got):
        by.setdefault((N, K), set()).add(p["split"])
    assert all(len(v) == 1 for v in by.values())   # a row's sums do not depend on how many rows there are


def test_the_largest(program):
    for s in ((2 ** 31 - 1, 1, 32, 0, 0), (1, 2 ** 31 - 1, 32, 0, 0), (2 ** 20, 2 ** 20, 32, 0, 0), (1, 1, 2 ** 30, 0, 0),
              (5, 7, 2 ** 30, 1, 0)):
        p = plans(program, [s])[0]
        assert p["ok"], s
        assert p["row_tiles"] > 0 and p["tok_tiles"] > 0
        check(s, p)


def test_sizes_of_the_tests_of_pairs(program):
    shapes = [(m, n, k, gated, 0) for m, n, k, gated in ref.PAIRS]
    rounds = set()
    for s, p in zip(shapes, plans(program, shapes)):
        assert p["faster"], s
        rounds.add((s[3], min(3, -(-p["row_tiles2"] * p["tok_tiles2"] // 76))))
    more = [(*s[:3], s[3], 0) for s in ref.PAIRS_SMALL]
    more += [(*s, gated, 0) for s in (ref.PAIRS_LARGEST, ref.PAIRS_GRAPH) for gated in (0, 1)]
    assert all(p["faster"] for p in plans(program, more))
    assert {(0, 1), (0, 2), (0, 3), (1, 1), (1, 2), (1, 3)} <= rounds
