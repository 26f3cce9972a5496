"""Host models of the synchronisation of speculative and branching decoding: the mbarrier protocol of the tree decode,
as sequences of barrier operations and of accesses to its buffers in the order of the kernel source, under random
schedules; and the order of a decode loop's kernels, launched as programmatic dependents of one another.  Mutations show
that the models notice what they are for."""
import random

import pytest

from tests.test_barrier_protocol import A, C, RD, RL, WR, W, Hazard, run
from tests.test_launch_order import Kernel, races
from tests.test_serve_protocol import append, host, one
from tests.test_serve_visibility import unseen


def tree_protocol(units, masked=None, active=(0, 1, 2, 3), slots=6, ring=16, descriptions=32, qexps=8, wait_pv=True,
                  wait_joined=True, wait_taken=True, wait_tile=True):
    """fa_decode_tree_kernel over units of the given step counts.  masked: the steps (of all) that are taken key by key, by
    default each unit's last; active: the softmax warps of a stream with rows.  The products, which run when the tensor cores
    come to them, are actors of their own."""
    steps = [(k, h, nh) for k, nh in enumerate(units) for h in range(nh)]
    total, last_of, n = len(steps), {}, 0
    for k, nh in enumerate(units):
        for s in (0, 1):  # the last step of each stream in the unit
            mine = [n + h for h in range(nh) if (n + h) & 1 == s]
            last_of[k, s] = mine[-1] if mine else None
        n += nh
    ends = {v for v in last_of.values() if v is not None}
    if masked is None:
        masked = {n for n, (k, h, nh) in enumerate(steps) if h + 1 == nh}
    end = len(units)

    def unit(k):
        return [(W, ("unit", k % descriptions), k // descriptions), (RD, ("slot", k % descriptions), k)]

    def over(k):
        return [(RL, ("slot", k % descriptions))]

    progs = {}
    # ---- copies
    g, n = [], 0
    for k, nh in enumerate(list(units) + [0]):
        g += [(WR, ("slot", k % descriptions), k, 19), (A, ("unit", k % descriptions))]
        for _ in range(nh):
            if n >= slots and wait_taken:
                g.append((W, ("taken", n % slots), n // slots - 1))
            g += [(WR, ("valid", n % slots), n, 1), (WR, ("rawbuf", n % slots), n, 5), (C, ("raw", n % slots))]
            n += 1
    progs["copies"] = g
    # ---- products: the warps that issue them, and the tensor cores
    qk, pv, tqk, tpv, n = [], [], [], [], 0
    for k, nh in enumerate(units):
        qk += unit(k) + [(W, "qfull", k)]
        pv += unit(k)
        for h in range(nh):
            s, t = n & 1, n & 3
            qk.append((W, ("full", 0, s), n >> 1))
            if n >= 4 and wait_pv:
                qk.append((W, ("pv", t), (n >> 2) - 1))
            qk.append((A, ("iqk", n)))
            tqk += [(W, ("iqk", n), 0)] + [(RD, ("tile", 0, s, c), n) for c in (0, 1)] + [(RD, ("Q", w), k) for w in range(8)]
            tqk += [(WR, ("S", t), n, len(active) + 1)] + [(RL, ("tile", 0, s, c)) for c in (0, 1)]
            tqk += [(A, ("s", t)), (A, ("kempty", s))]
            if h + 1 == nh:
                tqk += [(RL, ("Q", w)) for w in range(8)] + [(A, "qempty")]
            pv += [(W, ("full", 1, s), n >> 1), (W, ("p", t), n >> 2), (A, ("ipv", n))]
            tpv += [(W, ("ipv", n), 0)] + [(RD, ("tile", 1, s, c), n) for c in (0, 1)]
            tpv += [(RD, ("S", t), n), (WR, ("O", s), n, len(active) * (2 if n in ends else 1))]
            tpv += [(RL, ("tile", 1, s, c)) for c in (0, 1)] + [(RL, ("S", t)), (A, ("pv", t))]
            if h + 1 == nh:
                tpv.append((A, ("o", k & 3)))
            n += 1
        qk += over(k)
        pv += over(k)
    progs.update(qk=qk + unit(end) + over(end), pv=pv + unit(end) + over(end), tensor_qk=tqk, tensor_pv=tpv)

    def queries(w, k):
        # (s_qexp is read by the streams that have steps in the unit)
        readers = len(active) * sum(last_of[k, s] is not None for s in (0, 1))
        return [(WR, ("Q", w), k, 1), (WR, ("qexp", k % qexps, w), k, readers), (A, "qfull")]

    # ---- conversion
    for w in range(8):
        z, par, c = (w & 3) >> 1, w >> 2, w & 1
        g, n = [], 0
        for k, nh in enumerate(units):
            g += unit(k)
            hh, q = (n ^ par) & 1, k > 0
            while q or hh < nh:
                if hh < nh:
                    m = n + hh
                    g.append((W, ("info", m % ring), m // ring))
                    if z == 0 and m >= 2 and wait_tile:
                        g.append((W, ("kempty", par), (m >> 1) - 1))
                    if z == 1 and m >= 2 and wait_tile:
                        g.append((W, ("pv", (m - 2) & 3), (m - 2) >> 2))
                    g += [(RD, ("known", m % ring), m), (RD, ("rawbuf", m % slots), m)]
                    if z == 1 and m in masked:
                        g.append((WR, ("nan", par, c), m, len(active)))
                    g += [(WR, ("tile", z, par, c), m, 1), (RL, ("known", m % ring)), (RL, ("rawbuf", m % slots)),
                          (A, ("full", z, par)), (A, ("taken", m % slots))]
                if q:
                    q = False
                    g += [(W, "qempty", k - 1)] + queries(w, k)
                hh += 2
            n += nh
            g += over(k)
        progs[f"convert{w}"] = g + unit(end) + over(end)
    # ---- scout
    g = []
    for n, (k, h, nh) in enumerate(steps):
        g += unit(k) if h == 0 else []
        g += [(W, ("raw", n % slots), n // slots), (RD, ("rawbuf", n % slots), n), (RD, ("valid", n % slots), n),
              (WR, ("known", n % ring), n, 4 + len(active)), (RL, ("rawbuf", n % slots)), (RL, ("valid", n % slots)),
              (A, ("info", n % ring))]
        g += over(k) if h + 1 == nh else []
    progs["scout"] = g + unit(end) + over(end)
    # ---- softmax
    for w in range(8):
        s, r = w >> 2, w & 3
        on = r in active
        g, n0, posted = [(W, ("unit", 0), 0)], 0, False
        if units:
            g += queries(w, 0)
        for k, nh in enumerate(units):
            g += unit(k)
            first, noted = (s - n0) & 1, False
            for hh in range(first, nh, 2):
                n = n0 + hh
                g += [(W, ("s", n & 3), n >> 2), (W, ("info", n % ring), n // ring)]
                if on:
                    g += [(RD, ("S", n & 3), n), (RD, ("known", n % ring), n)]
                    if hh == first:
                        g += [(RD, ("qexp", k % qexps, x), k) for x in range(8)]
                        g += [(RL, ("qexp", k % qexps, x)) for x in range(8)]
                    if n in masked:
                        g += [(W, ("full", 1, n & 1), n >> 1)] + [(RD, ("nan", n & 1, c), n) for c in (0, 1)]
                        if posted and wait_joined:
                            g.append((W, "joined", k - 1))
                        posted = False
                        if not noted:
                            g.append((WR, ("row_nan", s, r), k, 2))
                        noted = True
                        g += [(RL, ("nan", n & 1, c)) for c in (0, 1)]
                    if hh >= 2:  # (O rescaled)
                        g += [(W, ("pv", (n - 2) & 3), (n - 2) >> 2), (RD, ("O", s), n - 2), (RL, ("O", s))]
                    g += [(RL, ("known", n % ring)), (RL, ("S", n & 3))]
                if posted and wait_joined:
                    g.append((W, "joined", k - 1))
                posted = False
                g.append((A, ("p", n & 3)))
            if posted and wait_joined:
                g.append((W, "joined", k - 1))
            g += [(WR, ("post", s, r), k, 2), (A, ("posted", s)), (W, ("posted", s ^ 1), k), (W, ("o", k & 3), k >> 2)]
            g += [(RD, ("post", x, r), k) for x in (0, 1)]
            if on:
                g += [(op, ("O", x), *(() if op == RL else (last_of[k, x],)))
                      for x in (0, 1) if last_of[k, x] is not None for op in (RD, RL)]
                for x in (0, 1):
                    if any(n in masked for n in range(n0, n0 + nh) if n & 1 == x):
                        g += [(RD, ("row_nan", x, r), k), (RL, ("row_nan", x, r))]
            g += [(RL, ("post", x, r)) for x in (0, 1)] + [(A, "joined")]
            posted = True
            n0 += nh
            g += over(k)
        progs[f"softmax{w}"] = g + unit(end) + over(end)
    counts = {"qfull": 8, "qempty": 1, "joined": 8}
    counts |= {("unit", i): 1 for i in range(descriptions)}
    counts |= {("raw", i): 1 for i in range(slots)} | {("taken", i): 4 for i in range(slots)}
    counts |= {("info", i): 1 for i in range(ring)}
    counts |= {("full", z, i): 2 for z in (0, 1) for i in (0, 1)} | {("kempty", i): 1 for i in (0, 1)}
    counts |= {("s", i): 1 for i in range(4)} | {("p", i): 4 for i in range(4)}
    counts |= {("pv", i): 1 for i in range(4)} | {("o", i): 1 for i in range(4)} | {("posted", i): 4 for i in (0, 1)}
    counts |= {(x, n): 1 for x in ("iqk", "ipv") for n in range(total)}
    return progs, counts


UNITS = [[], [1], [2], [5], [1] * 9, [3, 1, 4, 1, 5], [1, 9, 2], [2, 2, 2, 2, 2], [20], [1] * 36]


@pytest.mark.parametrize("active", [(0, 1, 2, 3), (0,)])
@pytest.mark.parametrize("units", UNITS, ids=str)
def test_tree_protocol(units, active):
    for seed in range(8):
        every = set(range(sum(units))) if seed % 2 else None  # (all steps key by key, or each unit's last)
        run(*tree_protocol(units, every, active), random.Random(seed))


def caught(units, **mutation):
    for seed in range(60):
        try:
            run(*tree_protocol(units, **mutation), random.Random(seed))
        except Hazard:
            return True
    return False


@pytest.mark.parametrize("units, mutation", [
    ([24], dict(ring=6)), ([1] * 12, dict(descriptions=3)), ([1] * 12, dict(qexps=1)), ([14], dict(wait_pv=False)),
    ([1] * 8, dict(wait_joined=False)), ([12], dict(wait_taken=False)), ([12], dict(wait_tile=False)),
], ids=lambda x: "-".join(x) if isinstance(x, dict) else str(len(x)))
def test_the_model_notices(units, mutation):
    assert caught(units, **mutation)


# --------------------------------------------------------------------------- launch order

def pages():
    return [one("pages", ("refs", "table", "lens", "source", "pages_ws"), ("refs", "table", "copies", "pages_ws"))]


def masks():
    return [one("mask", ("parents", "cu"), ("mask",))]


def layer(wait=True):
    """Copies of forked pages, the drafts' rows, their attention and merge, and the rows that are kept."""
    begin = [("wait",), ("trigger",)]
    att = Kernel("attention", begin + [("read", "q", "cache", "lens", "table", "mask", "cu"),
                                       ("write", "part", "cuts", "out", "lse_out")], pdl=True)
    merge = Kernel("merge", (begin if wait else [("trigger",)]) + [("read", "part", "cuts"), ("write", "out", "lse_out")],
                   pdl=True)
    return ([one("copies", ("copies", "cache"), ("cache",))] + append() + [att, merge] +
            [one("compaction", ("keep", "table", "cache"), ("cache",))])


INPUTS = ("q", "k", "v", "lens", "source", "parents", "cu", "keep")


def test_a_decode_loop_is_ordered():
    loop = []
    for _ in range(2):
        loop += [host("producer", (), INPUTS)] + pages() + masks() + layer() + layer()
        loop += [host("consumer", ("out", "lse_out", "cache", "table", "refs"), INPUTS + ("part", "cuts", "pages_ws"))]
    assert races(loop) == [] and unseen(loop) == []


def test_the_model_notices_a_merge_that_does_not_wait():
    bad = races([host("producer", (), INPUTS)] + layer(wait=False))
    assert ("attention", "write", "part", "merge", "read") in bad
