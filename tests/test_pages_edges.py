"""Copies, compaction and bookkeeping of pages at their edges, against the models of tests/test_pages.py."""
import numpy as np
import pytest
import torch

import exact_attention_25_gb300 as fa
from exact_attention_25_gb300 import _lib
from tests.test_pages import Pool, copied, host, ints, lists_of, pages, random_pages, run_compact, same, updated
from tests.test_serve_edges import checked  # noqa: F401 (a fixture)

gpu = pytest.mark.gpu


@gpu
@pytest.mark.parametrize("page", [16, 64, 1024])
def test_counts_of_rows_that_are_none(page):
    """Entries with the smallest numbers for rows do nothing, in any part of the page."""
    cache, guard = random_pages(8, 2, page, 64, 1)
    want = host(cache)
    copies = [[0, 1, -2 ** 31], [2, 3, -2 ** 31 + 16], [4, 5, -2 ** 31 + page], [6, 7, 9]]
    copied(want, want, copies)
    fa.cache_copy_pages(cache, cache, ints(copies).cuda())
    fa.fa_device_status()
    guard()
    same(cache, want)


@gpu
@pytest.mark.parametrize("room", [0, 5])
def test_a_step_without_slots(room):
    """No slots: nothing to copy, and the free pages are counted."""
    refs = ints([0, 2, 0, 0, 1, 0, 0]).cuda()
    table, none = torch.zeros(0, room, dtype=torch.int32).cuda(), torch.zeros(0, dtype=torch.int32).cuda()
    copies, counts = fa.pages_update(refs, table, none, none, none, none, 16)
    assert copies.shape == (0, 3) and counts.tolist() == [0, 5]
    out = torch.zeros(0, 3, dtype=torch.int32).cuda(), torch.full((2,), 9, dtype=torch.int32).cuda()
    fa.fa_pages_update(refs, table, none, none, none, none, 16, *out, torch.zeros(0, dtype=torch.uint8).cuda())
    fa.fa_device_status()
    assert out[1].tolist() == [0, 5] and refs.tolist() == [0, 2, 0, 0, 1, 0, 0]
    with pytest.raises(fa.FaError):
        fa.pages_update(refs, table, none, none, none, none, 24)


# ------------------------------------------------------------------------------ checked library

def pages_steps(slots=70, num_pages=600, most=12, page=16):
    """Steps in which sequences begin, fork, write on in shared pages, are trimmed and end, the last one with too few pages;
    what each leaves."""
    refs = torch.zeros(num_pages, dtype=torch.int32).cuda()
    table = torch.full((slots, most), -1, dtype=torch.int32).cuda()
    r, lens, out = np.random.RandomState(1), np.zeros(slots, np.int64), []
    for step in range(4):
        source = np.where(r.rand(slots) < 0.4, r.randint(-1, slots, slots), np.arange(slots))
        kept = np.where(source < 0, 0, np.maximum(lens[source] - r.randint(0, 9, slots), 0))
        new = np.minimum(kept + r.randint(0, 60, slots), most * page) if step < 3 else np.full(slots, most * page)
        copies, counts = fa.pages_update(refs, table, *(ints(x).cuda() for x in (lens, source, kept, new)), page)
        out += [copies, counts, refs.clone(), table.clone()]
        if step < 3:
            lens = new
    return out


@gpu
def test_checked_library_gives_the_same_pages(checked):  # noqa: F811
    with _lib.library(_lib.LIB_PATH):
        want = pages_steps()
        fa.fa_device_status()
    assert [c[0].item() > 0 for c in want[1::4]] == [False, False, False, True]
    with _lib.library(checked):
        got = pages_steps()
        fa.fa_device_status()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@gpu
def test_checked_library_catches_shrunk_extents_of_pages(checked):  # noqa: F811
    with _lib.library(checked) as lib:
        lib.fa_debug_set_flags(2)  # every extent one row short
        try:
            pages_steps()
            with pytest.raises(fa.FaError) as e:
                fa.fa_device_status()
            assert e.value.code == -9
        finally:
            lib.fa_debug_set_flags(0)
        pages_steps()
        fa.fa_device_status()


# ------------------------------------------------------------------------------ devices, sizes

@gpu
def test_clusters_of_eight_give_the_same_pages():
    """A device that holds no 16 CTAs in a cluster (a test hook) takes 8 for the same result."""
    lib = fa.load()
    want = pages_steps(500, 70000, 40)
    lib.fa_debug_set_flags(4)
    try:
        got = pages_steps(500, 70000, 40)
    finally:
        lib.fa_debug_set_flags(0)
    fa.fa_device_status()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@gpu
@pytest.mark.parametrize("share", [0.3, 0.9])
@pytest.mark.parametrize("B, rows, Hkv", [(1, 9000, 1), (2, 5000, 2), (1, 1300, 8), (40, 600, 8)])
def test_long_lists_of_short_rows(B, rows, Hkv, share):
    """Rows of 64: several steps to a sequence, with one thread block each and with several that wait for one another."""
    n = [rows - 7 * b for b in range(B)]
    run_compact(n, lists_of(n, share, B), [3 * b for b in range(B)], Hkv, 64, 64, 5)


@gpu
def test_more_slots_than_a_cluster_takes_at_once():
    """20000 slots, 1250 to a thread block, which takes 1024 at once."""
    slots, page, most = 20000, 16, 80
    r = np.random.RandomState(3)
    pool = Pool(60000, slots, pages(most, page), page)
    for step in range(4):
        source = np.arange(slots)
        move = r.rand(slots)
        source[move < 0.3] = r.randint(0, slots, (move < 0.3).sum())
        source[move < 0.1] = -1
        kept = [0 if s < 0 else max(pool.lens[s] - int(r.choice([0, 0, 1, 3, 20])), 0) for s in source]
        grow = most if step == 2 else 25
        new = [min(k + int(r.choice([0, 1, 5, grow])), most) for k in kept]
        if step == 2:
            new = [most] * slots  # 100000 pages
        counts, copies = pool.step(source.tolist(), kept, new)
        assert (counts[0] > 0) == (step == 2)
        assert step != 1 or (copies[:, 0] >= 0).sum() > 1000


@gpu
@pytest.mark.parametrize("short", [False, True])
def test_rows_of_a_table_wider_than_a_batch(short):
    """12 slots of 2^27 entries, of which 8 are taken at once; entries beyond 2^31 bytes; the far ones stay as they are."""
    slots, M, page, num = 12, 2 ** 27, 16, 400
    table = torch.full((slots, M), -1, dtype=torch.int32, device="cuda")
    table[:, 64:] = -7
    refs = torch.zeros(num, dtype=torch.int32).cuda()
    r = np.random.RandomState(2)
    lens, t, c = [0] * slots, np.full((slots, 64), -1), np.zeros(num, np.int64)
    for step in range(3):
        source = np.where(r.rand(slots) < 0.5, r.randint(-1, slots, slots), np.arange(slots)).tolist()
        kept = [0 if s < 0 else max(lens[s] - int(r.randint(0, 20)), 0) for s in source]
        new = [k + int(r.randint(0, 150)) for k in kept]
        if short and step == 2:
            new = [900] * slots
        got = fa.pages_update(refs, table, *(ints(x).cuda() for x in (lens, source, kept, new)), page)
        fa.fa_device_status()
        c, t, copies, counts = updated(c, t, lens, source, kept, new, page)
        assert got[1].tolist() == counts and (got[0].cpu().numpy() == copies).all()
        assert (table[:, :64].cpu().numpy() == t).all() and (refs.cpu().numpy() == c).all()
        assert (counts[0] > 0) == (short and step == 2)
        lens = lens if counts[0] else new
    assert (table[:, 64:] == -7).all()
