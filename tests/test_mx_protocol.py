"""The waits of the kernel of the MXFP4 products (csrc/mx_product.cu), on the CPU: its warps as
they fill and use the ring of stages, under random schedules.  A wait for a barrier is told a
phase by its parity alone, so one that is two phases off returns at once; on the GPU such a
mistake can fault.  Here it is an assertion, as is an arrival more than a barrier counts."""
import os
import random

import pytest


class Barrier:
    def __init__(self, count):
        self.count, self.pending, self.tx, self.phase = count, count, 0, 0

    def _look(self):
        if self.pending == 0 and self.tx == 0:
            self.phase, self.pending = self.phase + 1, self.count

    def arrive(self, tx=0):
        assert self.pending > 0, "more arrivals than the barrier counts"
        self.tx, self.pending = self.tx + tx, self.pending - 1
        self._look()

    def complete(self):
        self.tx -= 1
        self._look()

    def ready(self, parity):
        return (self.phase & 1) != parity


def wait(bar, parity, meant):
    while not bar.ready(parity):
        yield
    assert bar.phase == meant, f"a wait for phase {meant} returned in phase {bar.phase}"
    yield


def play(rng, procs, later):
    speed = [rng.choice([0.02, 0.3, 1, 5]) for _ in procs]
    idle = 0
    while procs or later:
        if later and (not procs or rng.random() < rng.choice([0.05, 0.5])):
            later.pop(0)()
            idle = 0
            continue
        i = rng.choices(range(len(procs)), speed)[0]
        try:
            next(procs[i])
        except StopIteration:
            procs.pop(i), speed.pop(i)
            idle = 0
        idle += 1
        assert idle < 2000000, "no warp gets any further"


def run(rng, S, k0, k1, tiles, gated, pair, fp16, tma, turns=True, loaders=4, tma_warps=2, out=8):
    """One block's roles over its tiles; k0 .. k1: its steps of K."""
    weights, steps = 2 if gated else 1, k1 - k0
    moves = tma or not fp16                       # TMA brings something
    full = [Barrier(1 + (not tma) + moves) for _ in range(S)]
    empty = [Barrier(weights) for _ in range(S)]
    acc_full = [Barrier(2 if gated or pair else 1) for _ in range(2)]
    acc_empty = [Barrier(out) for _ in range(2)]
    rows = [Barrier(1) for _ in range(steps)]
    turn = [Barrier(1) for _ in range(loaders)]
    later = []                                    # what the hardware does by itself, in order

    def codes(me):
        for g in range(me, tiles * steps, tma_warps):
            s, use = g % S, g // S
            if use > 0:
                yield from wait(empty[s], (use - 1) & 1, use)
            if moves:
                full[s].arrive(tx=1)
                later.append(full[s].complete)
            yield
            if not tma:
                later.append(full[s].arrive)
                yield

    def scales(me):
        q0 = k0 >> 2
        groups = ((k1 - 1) >> 2) - q0 + 1
        for g in range(me, tiles * groups, loaders):
            t, q = divmod(g, groups)
            first, last = max(k0, 4 * (q0 + q)), min(k1, 4 * (q0 + q) + 4)
            yield
            if g > 0 and turns:
                yield from wait(turn[me], (g // loaders - (me == 0)) & 1, g // loaders + (me != 0))
            done, written = t * steps + first - k0, []
            for k in range(first, last):
                s, use = done % S, done // S
                if use > 0:
                    yield from wait(empty[s], (use - 1) & 1, use)
                if k == last - 1 and turns:
                    turn[(me + 1) % loaders].arrive()
                    yield
                assert full[s].phase == use
                written.append(s)
                done += 1
                if k == last - 1 or k & 3 == 3 or (k & 3 == 1 and S < 8):
                    yield
                    for s in written:
                        full[s].arrive()
                        yield
                    written = []

    def products(me):
        if not (gated or pair or me == 0):
            return
        g = 0
        for n in range(tiles):
            if n >= 2:
                yield from wait(acc_empty[n & 1], ((n >> 1) - 1) & 1, n >> 1)
            for k in range(steps):
                if gated or not pair or g & 1 == me:
                    s, use = g % S, g // S
                    while fp16 and n == 0 and not rows[k].ready(0):
                        yield
                    yield from wait(full[s], use & 1, use + 1)
                    later.append(empty[s].arrive)
                    yield
                g += 1
            later.append(acc_full[n & 1].arrive)
            yield

    def results(me):
        for k in range(me, steps if fp16 else 0, out):
            rows[k].arrive()
            yield
        for n in range(tiles):
            yield from wait(acc_full[n & 1], (n >> 1) & 1, (n >> 1) + 1)
            acc_empty[n & 1].arrive()
            yield

    procs = ([scales(i) for i in range(loaders)] + [products(i) for i in range(2)] +
             [results(i) for i in range(out)] + [codes(i) for i in range(tma_warps)])
    play(rng, procs, later)


def run_pair(rng, S, steps, tiles, two, turns=True, loaders=4, tma_warps=2, out=8):
    """Two blocks that share their tiles (csrc/mx_pair.cu)."""
    full = [[Barrier(3 - rank) for _ in range(S)] for rank in range(2)]
    empty = [[Barrier(1) for _ in range(S)] for _ in range(2)]
    acc_full = [[Barrier(2 if two else 1) for _ in range(2)] for _ in range(2)]
    acc_empty = [Barrier(2 * out) for _ in range(2)]              # of the one that issues
    turn = [[Barrier(1) for _ in range(loaders)] for _ in range(2)]
    later = []

    def both(bars):
        for b in bars:
            b.arrive()

    def codes(rank, me):
        for g in range(me, tiles * steps, tma_warps):
            s, use = g % S, g // S
            if use > 0:
                yield from wait(empty[rank][s], (use - 1) & 1, use)
            full[rank][s].arrive(tx=1)
            later.append(full[rank][s].complete)
            yield

    def scales(rank, me):
        groups = (steps + 3) // 4
        for g in range(me, tiles * groups, loaders):
            t, q = divmod(g, groups)
            last = min(steps, 4 * q + 4)
            yield
            if g > 0 and turns:
                yield from wait(turn[rank][me], (g // loaders - (me == 0)) & 1, g // loaders + (me != 0))
            done, written = t * steps + 4 * q, []
            for k in range(4 * q, last):
                s, use = done % S, done // S
                if use > 0:
                    yield from wait(empty[rank][s], (use - 1) & 1, use)
                if k == last - 1 and turns:
                    turn[rank][(me + 1) % loaders].arrive()
                    yield
                assert full[rank][s].phase == use
                written.append(s)
                done += 1
                if k == last - 1 or k & 3 == 3 or (k & 3 == 1 and S < 8):
                    yield
                    for s in written:
                        full[rank][s].arrive()
                        yield
                    written = []

    def products(me):
        if me and not two:
            return
        g = 0
        for n in range(tiles):
            if n >= 2:
                yield from wait(acc_empty[n & 1], ((n >> 1) - 1) & 1, n >> 1)
            for _ in range(steps):
                s, use = g % S, g // S
                if not two or g & 1 == me:
                    yield from wait(full[0][s], use & 1, use + 1)
                    assert full[1][s].phase == use + 1            # the other's operands are there
                    later.append(lambda s=s: both([empty[0][s], empty[1][s]]))
                    yield
                g += 1
            later.append(lambda n=n: both([acc_full[0][n & 1], acc_full[1][n & 1]]))
            yield

    def hand_on(me):
        for g in range(me, tiles * steps, 2):
            yield from wait(full[1][g % S], (g // S) & 1, g // S + 1)
            full[0][g % S].arrive()
            yield

    def last_uses(rank, me, before):
        yield from before
        alone = rank == 0 and not two
        for g in range(max(0, tiles * steps - S), tiles * steps)[::-1]:
            if (me == 0 if alone else g & 1 == me):
                yield from wait(empty[rank][g % S], (g // S) & 1, g // S + 1)

    def results(rank):
        for n in range(tiles):
            yield from wait(acc_full[rank][n & 1], (n >> 1) & 1, (n >> 1) + 1)
            if n + 2 < tiles:
                acc_empty[n & 1].arrive()
            yield

    procs = [last_uses(rank, me, job(me)) for rank, job in enumerate((products, hand_on)) for me in range(2)]
    for rank in range(2):
        procs += ([scales(rank, i) for i in range(loaders)] + [codes(rank, i) for i in range(tma_warps)] +
                  [results(rank) for _ in range(out)])
    play(rng, procs, later)
    for b in [*full[0], *full[1], *empty[0], *empty[1]]:          # nothing is left half arrived
        assert b.pending == b.count and b.tx == 0
    for b in acc_empty:
        assert b.pending == b.count


def draw(rng):
    mode, k0 = rng.choice(["plain", "pair", "gated", "fp16"]), rng.randint(0, 9)
    return dict(k0=k0, k1=k0 + rng.randint(1, 30), tiles=rng.randint(1, 6), gated=mode == "gated",
                pair=mode in ("pair", "fp16"), fp16=mode == "fp16", tma=rng.random() < 0.6)


@pytest.mark.parametrize("seed", range(6))
def test_every_wait_is_for_its_phase(seed):
    rng = random.Random(seed)
    for _ in range(40):
        run(rng, 2 * rng.randint(2, 8), **draw(rng))


@pytest.mark.parametrize("seed", range(4))
def test_pairs_of_blocks(seed):
    rng = random.Random(100 + seed)
    for _ in range(8):
        run_pair(rng, 2 * rng.randint(2, 8), rng.randint(1, 20), rng.randint(1, 5), rng.random() < 0.5)
    with pytest.raises(AssertionError):
        for _ in range(100):
            run_pair(rng, 2 * rng.randint(2, 8), rng.randint(8, 30), rng.randint(1, 6), rng.random() < 0.5, turns=False)


@pytest.mark.parametrize("wrong", ["no turns", "odd stages"])
def test_the_schedules_find_what_is_wrong(wrong):
    """Without the loaders' turns, or with an odd number of stages, some schedule goes wrong."""
    rng = random.Random(1)
    with pytest.raises(AssertionError):
        for _ in range(200):
            run(rng, 2 * rng.randint(2, 8) + (wrong == "odd stages"), turns=wrong != "no turns", **draw(rng))


def test_order_of_the_kernel_of_pairs():
    """Tensor memory is taken behind the wait for the kernel before, and the next one is let in
    behind that; it is freed when both blocks are done."""
    import bit_group_quantized_qgemv_gb300 as q
    with open(os.path.join(os.path.dirname(q.__file__), "csrc", "mx_pair.cu")) as f:
        body = f.read().split("mx_pair_kernel(", 1)[1].split("cudaError_t launch(", 1)[0]
    order = [body.index(s) for s in ("pdl_wait()", "tc::alloc_pair(", "pdl_launch_dependents()", "  // neither block ends",
                                     "tc::dealloc_pair(")]
    assert order == sorted(order) and body.rindex("cluster_wait()") < order[-1]
    assert body.count("tc::alloc_pair(") == body.count("pdl_wait()") == body.count("tc::dealloc_pair(") == 1
