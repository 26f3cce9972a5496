"""Copies, compaction and bookkeeping of pages at their edges, against the models of tests/test_pages.py."""
import numpy as np
import pytest
import torch

import exact_attention_25_gb300 as fa
from tests.test_pages import copied, host, ints, random_pages, same

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
