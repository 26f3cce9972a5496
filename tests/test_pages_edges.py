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
