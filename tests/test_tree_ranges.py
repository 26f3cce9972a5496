"""Attention of drafted trees over value rows of every size that the cache holds."""
import numpy as np
import pytest
import torch

import exact_attention_25_gb300 as fa
from tests.test_cache import cu, table_for
from tests.test_decode_cache import _check, random_cache, to_cache
from tests.tree_util import ancestors, tree_reference, words_of

gpu = pytest.mark.gpu


def ints(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32)


def run(a, ctas, scale):
    q, codes, exps, mask, nq, nk, table = a
    got = fa.forward_decode_tree(q.cuda(), to_cache(codes, exps), mask.cuda(), cu([nq]).cuda(), ints([nk]).cuda(),
                                 table.cuda(), nq, nk, scale, None, ctas)
    fa.fa_device_status()
    return got


def check(a, b, ctas, scale, what=""):
    q, _, _, mask, nq, nk, table = a
    codes, plain, page = b
    got = run(a, ctas, scale)
    _check(got, tree_reference(q, codes, plain, table, [nq], [nk], [nk - nq], mask, page, scale), what)


@gpu
@pytest.mark.parametrize("ctas", [2, 4])
@pytest.mark.parametrize("d", [64, 128])
def test_parts_whose_weights_are_tiny(d, ctas):
    """Keys 2^-160 of the others' weight with values 2^175 times their size, in parts of their own: what they add is of the
    result's size, although a part's weight is below fp32's smallest."""
    nk, page = 128 * 12, 64
    table, pool = table_for([nk], page, 0, 1)
    codes, exps = random_cache(pool, 1, page, d, 1)
    codes[1] &= 0xBF
    codes[0] = 0x38  # 1
    exps[0], exps[1] = 127, 127 - 105
    for j in range(4 * 128):  # (two thread blocks: the first has four of the twelve blocks of keys)
        at = int(table[0, j // page]), slice(None), j % page
        codes[0][at], exps[1][at] = 0, 127 + 70
    scale = 160 * float(np.log(2.0)) / d
    q, mask = torch.ones(2, 1, d).bfloat16(), words_of(ancestors([-1, 0]), 1)
    check((q, codes, exps, mask, 2, nk, table), (codes, exps, page), ctas, scale)
