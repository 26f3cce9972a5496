"""Host models of the serving kernels' synchronisation: the mbarrier protocols of the decode over
the cache and of the decode with shared prefixes, as sequences of barrier operations in the order of
the kernel source, under random schedules; and the order of the serving calls' kernels, launched as
programmatic dependents of one another.  Mutations show that the models notice what they are for."""
import random

import pytest

from tests.test_barrier_protocol import A, C, RD, RL, WR, W, Hazard, run
from tests.test_launch_order import Kernel, races

SEEDS = range(40)


# --------------------------------------------------------------------------- shared prefixes

def shared_protocol(units, st=3, slots=8, two_s=True, wait_p=True, release_q_early=False):
    """fa_decode_shared_kernel over units of the given block counts (its share): producer (warp 4),
    MMA issuer (warp 5), four softmax warps.  The last block of every unit waits for V
    itself, to clear rows.  S, O, Q and the unit descriptions are tracked as buffers."""
    sb = (lambda n: n & 1) if two_s else (lambda n: 0)
    sph = (lambda n: n >> 1) if two_s else (lambda n: n)
    prod, mma, n = [], [], 0

    def load_v(i):
        return ([(W, ("vempty", i % st), i // st - 1)] if i >= st else []) + [(C, ("vfull", i % st))]

    for k, J in enumerate(list(units) + [0]):
        prod += [(WR, ("slot", k % slots), k, 5), (A, ("unit", k % slots), k // slots)]
        for j in range(J):
            if j == 0:
                if k > 0:
                    prod.append((W, "qempty", k - 1))
                prod += [(WR, "Q", k, 1), (C, "qfull")]
            if n >= st:
                prod.append((W, ("kempty", n % st), n // st - 1))
            prod.append((C, ("kfull", n % st)))
            if n > 0:
                prod += load_v(n - 1)
            n += 1
        if J == 0 and n > 0:  # the last V goes out before the end is announced
            prod[-2:-2] = load_v(n - 1)
    blocks = [(k, j, J) for k, J in enumerate(units) for j in range(J)]

    def new_unit(k):
        return [(W, ("unit", k % slots), k // slots), (RD, ("slot", k % slots), k), (RL, ("slot", k % slots))]

    def issue_s(n):
        if n == len(blocks):
            return new_unit(len(units))
        k, j, J = blocks[n]
        out = []
        if j == 0:
            out += new_unit(k) + [(W, "qfull", k)]
        out += [(W, ("kfull", n % st), n // st), (WR, ("S", n & 1), n, 4), (RD, "Q", k),
                (C, ("sfull", sb(n))), (C, ("kempty", n % st))]
        if j + 1 == J or release_q_early:
            out += ([(RL, "Q")] if j + 1 == J else []) + [(C, "qempty")] * (j + 1 == J or j == 0)
        return out

    mma += issue_s(0)
    for n, (k, j, J) in enumerate(blocks):
        mma += issue_s(n + 1) + ([(W, "pfull", n)] if wait_p else []) + [(W, ("vfull", n % st), n // st)]
        if j == 0:
            mma.append((WR, "O", k, 4))
        mma += [(C, "pv"), (C, ("vempty", n % st))]
    progs = {"producer": prod, "mma": mma}
    for w in range(4):
        g, n = [], 0
        for k, J in enumerate(units):
            g += [(W, ("unit", k % slots), k // slots), (RD, ("slot", k % slots), k)]
            for j in range(J):
                g += [(W, ("sfull", sb(n)), sph(n)), (RD, ("S", n & 1), n), (RL, ("S", n & 1))]
                if j + 1 == J:
                    g.append((W, ("vfull", n % st), n // st))
                if j > 0:
                    g.append((W, "pv", n - 1))
                g.append((A, "pfull", n))
                n += 1
            g += [(W, "pv", n - 1), (RD, "O", k), (RL, "O"), (RL, ("slot", k % slots))]
        k = len(units)
        g += [(W, ("unit", k % slots), k // slots), (RD, ("slot", k % slots), k), (RL, ("slot", k % slots))]
        progs[f"softmax{w}"] = g
    counts = {"qfull": 1, "qempty": 1, "pfull": 4, "pv": 1}
    counts |= {("unit", i): 1 for i in range(slots)}
    counts |= {("sfull", i): 1 for i in (0, 1)}
    counts |= {(x, i): 1 for x in ("kfull", "kempty", "vfull", "vempty") for i in range(st)}
    return progs, counts


UNITS = [[], [1], [2], [5], [1, 1, 1, 1, 1, 1, 1, 1, 1, 1, 1, 1], [3, 1, 4, 1, 5], [1, 7, 2],
         [2, 2, 2, 2, 2, 2, 2, 2, 2, 2]]


@pytest.mark.parametrize("st", [3, 6])  # d = 128 and d = 64
@pytest.mark.parametrize("units", UNITS)
def test_shared_protocol(units, st):
    for seed in SEEDS:
        run(*shared_protocol(units, st), random.Random(seed))


def caught(make):
    for seed in range(400):
        try:
            run(*make(), random.Random(seed))
        except Hazard:
            return True
    return False


def test_the_model_notices_two_scores_on_one_barrier():
    assert caught(lambda: shared_protocol([6], two_s=False))


def test_the_model_notices_weights_that_are_not_waited_for():
    assert caught(lambda: shared_protocol([1] * 6, wait_p=False))


def test_the_model_notices_too_few_descriptions():
    assert caught(lambda: shared_protocol([1] * 12, slots=2))


def test_the_model_notices_queries_released_before_their_last_use():
    assert caught(lambda: shared_protocol([3, 3, 3], release_q_early=True))


# --------------------------------------------------------------------------- decode over the cache

def cache_protocol(units, st=3, row_tiles=1, slots=8, rounds_per_unit=1, wait_taken=True):
    """fa_decode_cache_kernel: the copying warp and four compute warps, which hand their sums over
    at the end of each unit (rounds_per_unit: 8-row tiles of a warp)."""
    prod, it = [], 0
    for k, J in enumerate(list(units) + [0]):
        prod += [(WR, ("slot", k % slots), k, 4), (A, ("unit", k % slots), k // slots)]
        for _ in range(J):
            if it >= st:
                prod.append((W, ("empty", it % st), it // st - 1))
            prod += [(WR, ("stage", it % st), it, 4), (C, ("full", it % st))]
            it += 1
    progs = {"copies": prod}
    ns = 4 // row_tiles
    for w in range(4):
        slot = w // row_tiles
        g, it, rounds = [], 0, 0
        for k, J in enumerate(list(units) + [0]):
            g += [(W, ("unit", k % slots), k // slots), (RD, ("slot", k % slots), k)]
            for _ in range(J):
                s = it % st
                g += [(W, ("full", s), it // st), (RD, ("stage", s), it), (RL, ("stage", s)), (A, ("empty", s))]
                it += 1
            for n in range(rounds_per_unit if J else 0):
                half = ns // 2
                while half > 0:
                    x = 2 if half == 1 and ns == 4 else w & 1
                    if slot < 2 * half:
                        if slot >= half:
                            if rounds > 0 and wait_taken:
                                g.append((W, ("taken", x), rounds - 1))
                            g += [(WR, ("xch", x), rounds, 1), (A, ("given", x))]
                        else:
                            g += [(W, ("given", x), rounds), (RD, ("xch", x), rounds),
                                  (RL, ("xch", x)), (A, ("taken", x))]
                    half //= 2
                rounds += 1
            g.append((RL, ("slot", k % slots)))
        progs[f"warp{w}"] = g
    counts = {("unit", i): 1 for i in range(slots)}
    counts |= {("full", i): 1 for i in range(st)} | {("empty", i): 4 for i in range(st)}
    counts |= {(x, i): 1 for x in ("given", "taken") for i in range(3)}
    return progs, counts


@pytest.mark.parametrize("row_tiles, rounds", [(1, 1), (1, 2), (2, 2), (4, 2)])
@pytest.mark.parametrize("st", [3, 6])
@pytest.mark.parametrize("units", UNITS)
def test_cache_protocol(units, st, row_tiles, rounds):
    for seed in SEEDS:
        run(*cache_protocol(units, st, row_tiles, rounds_per_unit=rounds), random.Random(seed))


def test_the_model_notices_sums_that_are_overwritten():
    assert caught(lambda: cache_protocol([1] * 4, wait_taken=False, rounds_per_unit=2))


def test_the_model_notices_too_few_descriptions_of_the_cache_decode():
    assert caught(lambda: cache_protocol([1] * 20, st=6, slots=3))


# --------------------------------------------------------------------------- launch order

def one(name, reads, writes):
    """A kernel that waits, lets the next one start and then works."""
    return Kernel(name, [("wait",), ("trigger",), ("read",) + reads, ("write",) + writes], pdl=True)


def rope():
    return [one("rope", ("q", "k", "pos"), ("q", "k"))]


def append():
    return [one("append", ("k", "v", "lens", "table"), ("cache",))]


def decode(early_wait=True, trigger_first=False):
    """The attention kernel, and the merge, which reads the lengths before its own wait."""
    begin = [("trigger",), ("wait",)] if trigger_first else [("wait",), ("trigger",)]
    att = Kernel("attention", begin + [("read", "q", "cache", "lens", "table"), ("write", "part", "out", "lse_out")],
                 pdl=True)
    merge = Kernel("merge", [("read", "lens")] + ([("wait",)] if early_wait else []) +
                   [("trigger",), ("read", "part"), ("write", "out", "lse_out")], pdl=True)
    return [att, merge]


def host(name, reads, writes):
    return Kernel(name, [("read",) + reads, ("write",) + writes], pdl=False)


def early(name, reads, writes):
    """Another program's kernel that triggers before it writes."""
    return Kernel(name, [("trigger",), ("wait",), ("read",) + reads, ("write",) + writes], pdl=True)


STEP = ("q", "k", "v", "pos", "lens", "table")


def test_serving_steps_are_ordered():
    for first in (host, early):
        steps = []
        for _ in range(3):
            steps += [first("producer", (), STEP)] + rope() + append() + decode()
        assert races(steps + decode() + [host("consumer", ("out", "lse_out", "cache"), STEP + ("part",))]) == []


def test_the_model_notices_a_merge_that_does_not_wait():
    bad = races([host("producer", (), STEP)] + decode(early_wait=False))
    assert ("attention", "write", "part", "merge", "read") in bad


def test_the_model_notices_an_attention_kernel_that_triggers_before_its_wait():
    # its merge would read the lengths while the kernel before still writes them
    bad = races([early("producer", (), STEP)] + decode(trigger_first=True))
    assert ("producer", "write", "lens", "merge", "read") in bad
