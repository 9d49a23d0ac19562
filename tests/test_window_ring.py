"""The barriers of the D = 128 window forward's K and V rings, on the CPU.

A model of the producer, the product issuer and the asynchronous copies runs the
kernel's order of waits and releases under random schedules.  A wait by parity
sees only whether the barrier's phase has the other parity, so a slot may be
released for a step only after that step's tile is known to have arrived:
released earlier, a phase can complete twice before the producer looks, and its
wait then never ends.  Where the idle Q tile releases V is read from the source."""
import os
import random

import pytest

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "tiled_memory_efficient_gb300",
                      "csrc", "attn_fwd.cu")
KS, VS = 2, 3   # K and V slots


def idle_release_after_product():
    """Does the issuer release V for an idle tile 0 after tile 1's product, which waits for V?"""
    text = open(SOURCE).read()
    loop = text[text.index("window_fwd_kernel(const"):]
    loop = loop[loop.index("for (int j = 0; j < steps; ++j)"):loop.index("g0 += steps;")]
    assert loop.count("mma_commit_elect(&v_empty[2 * vs]);") == 1 and loop.count("issue_pv(1, g") == 1
    return loop.index("mma_commit_elect(&v_empty[2 * vs]);") > loop.index("issue_pv(1, g")


class Barrier:
    def __init__(self):
        self.phase = 0       # phases completed; one arrival each

    def arrive(self):
        self.phase += 1

    def passed(self, parity):
        return (self.phase & 1) != parity


class Rings:
    def __init__(self):
        self.k_full, self.v_full = ([Barrier() for _ in range(n)] for n in (KS, VS))
        self.k_empty, self.v_empty = ([Barrier() for _ in range(2 * n)] for n in (KS, VS))
        self.pending = []      # barriers whose copy is on its way


def producer(r, units):
    g = 0
    for n0, n1, _ in units:
        for _ in range(max(n0, n1)):
            for n, full, empty in ((KS, r.k_full, r.k_empty), (VS, r.v_full, r.v_empty)):
                slot, parity = g % n, ((g // n) & 1) ^ 1
                for t in range(2):
                    while not empty[2 * slot + t].passed(parity):
                        yield False
                    yield True
                r.pending.append(full[slot])
                yield True
            g += 1


def issuer(r, units, after):
    """The order of window_fwd_kernel's issuing warp (its products complete at once: later
    only widens the distance to the producer)."""
    def wait(bars, n, g):
        while not bars[g % n].passed((g // n) & 1):
            yield False
        yield True

    def scores(t, g):
        yield from wait(r.k_full, KS, g)
        r.k_empty[2 * (g % KS) + t].arrive()

    def product(t, g):
        yield from wait(r.v_full, VS, g)
        r.v_empty[2 * (g % VS) + t].arrive()
    g0, ahead = 0, False
    for k, (n0, n1, x1) in enumerate(units):
        steps = max(n0, n1)
        after_x = lambda j: j + 2 if j + 1 == x1 else j + 1
        if not ahead:
            yield from scores(0, g0)
        ahead = False
        if n1 > 0:
            yield from scores(1, g0 + after_x(-1))
        for j in range(steps):
            g = g0 + j
            if j < n0:
                yield from product(0, g)
                if j + 1 < n0:
                    yield from scores(0, g + 1)
            else:
                r.k_empty[2 * (g % KS)].arrive()
                if not after:
                    r.v_empty[2 * (g % VS)].arrive()
                if j + 1 == steps and k + 1 < len(units):
                    yield from scores(0, g + 1)
                    ahead = True
            if j < n1 and j != x1:
                yield from product(1, g)
                if j >= n0 and after:
                    r.v_empty[2 * (g % VS)].arrive()
                if after_x(j) < n1:
                    yield from scores(1, g0 + after_x(j))
            else:
                r.k_empty[2 * (g % KS) + 1].arrive()
                r.v_empty[2 * (g % VS) + 1].arrive()
        g0 += steps


def runs_to_its_end(units, after, seed):
    rng = random.Random(seed)
    r = Rings()
    roles = [producer(r, units), issuer(r, units, after)]
    slow = rng.choice([0.02, 0.2, 0.5])       # how often the producer gets a turn
    stuck = 0
    while roles:
        if r.pending and rng.random() < 0.5:
            r.pending.pop(rng.randrange(len(r.pending))).arrive()
            stuck = 0
            continue
        i = 0 if len(roles) == 1 or rng.random() < slow else 1
        try:
            stuck = 0 if next(roles[i]) else stuck + 1
        except StopIteration:
            roles.pop(i)
        if stuck > 2000:
            return False
    return True


def _units(rng):
    out = []
    for _ in range(rng.randint(1, 5)):
        n0 = rng.randint(1, 5)
        n1 = rng.choice([0, n0, n0 + 1, n0 + 1])       # no rows, an even split, the usual one more
        out.append((n0, n1, rng.randrange(n0) if n1 > 1 and rng.random() < 0.5 else -1))
    return out


def test_the_model_finds_a_release_that_comes_too_early():
    rng = random.Random(1)
    assert not all(runs_to_its_end(_units(rng), False, s) for s in range(300))


@pytest.mark.parametrize("seed", range(4))
def test_every_schedule_of_the_kernels_order_ends(seed):
    rng, after = random.Random(seed), idle_release_after_product()
    for s in range(300):
        units = _units(rng)
        assert runs_to_its_end(units, after, s), (units, s)
