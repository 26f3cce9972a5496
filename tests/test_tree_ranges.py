"""Attention of drafted trees over value rows of every size that the cache holds (scales of 2^-110 to 2^120, rows of
zeros): the softmax's sum and lse do not depend on V, so steps of 64 keys whose rows lie hundreds of binades apart count
alike, in one stream and across both, and in parts that are merged."""
import numpy as np
import pytest
import torch

import exact_attention_25_gb300 as fa
from tests.test_cache import cu, table_for
from tests.test_decode_cache import _check, random_cache, to_cache
from tests.tree_util import ancestors, random_tree, tree_reference, words_of

gpu = pytest.mark.gpu
STEP = 64   # keys that are taken at once
ZERO = None  # a step of value rows of zeros


def ints(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32)


def batch(pattern, d, seed, spread=0, logits=1.0, nq=9, H=4, Hkv=2, page=64, steps=6):
    """A sequence whose value rows have the scales 2^pattern[step], cyclically, and codes below 2 in size; the tree is at its
    end.  Returns the call's arguments and the reference's."""
    nk = STEP * max(steps, len(pattern)) - 11
    table, pool = table_for([nk], page, 1, seed)
    codes, exps = random_cache(pool, Hkv, page, d, seed)
    codes[1] &= 0xBF
    r = np.random.RandomState(seed)
    plain = exps.copy()  # (for the reference's bounds: rows of zeros count as the smallest)
    small = min([e for e in pattern if e is not ZERO] + [0])
    for j in range(nk):
        e = pattern[j // STEP % len(pattern)]
        at = int(table[0, j // page]), slice(None), j % page
        if e is ZERO:
            codes[1][at] = np.where(r.rand(Hkv, d) < 0.5, 0, 0x80)
            exps[1][at], plain[1][at] = 127, 127 + small
        else:
            exps[1][at] = plain[1][at] = 127 + np.clip(e - r.randint(0, spread + 1, Hkv), -110, 120)
    q = (logits * torch.randn(nq, H, d, generator=torch.Generator().manual_seed(seed))).bfloat16()
    mask = words_of(ancestors(random_tree(r, nq)), 1)
    return (q, codes, exps, mask, nq, nk, table), (codes, plain, page)


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
@pytest.mark.parametrize("ctas", [1, 2])
@pytest.mark.parametrize("spread", [0, 3])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("e", [-110, -101, 0, 99, 114, 118, 120])
def test_all_rows_of_one_size(e, d, spread, ctas):
    a, b = batch([e], d, 3, spread, steps=24)
    check(a, b, ctas, d ** -0.5)


APART = {
    "zero_then_large": [ZERO, 40, ZERO, 40],
    "large_then_zero": [40, ZERO, 40, ZERO],
    "zero_first_in_both": [ZERO, ZERO, 40, 40],
    "large_first_in_both": [40, 40, ZERO, ZERO],
    "rising": [-110, -60, -10, 30, 80, 120],
    "falling": [120, 80, 30, -10, -60, -110],
    "streams_apart": [120, -110],
    "streams_apart_other": [-110, 120],
    "all_kinds": [0, 100, ZERO, -100, 60, -60, ZERO],
    "only_zeros": [ZERO],
    "zeros_and_the_smallest": [ZERO, -110, ZERO, -110, -110, ZERO],
}


@gpu
@pytest.mark.parametrize("logits", [0.0, 1.0, 20.0])
@pytest.mark.parametrize("ctas", [1, 3])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("case", list(APART))
def test_steps_of_very_different_size(case, d, ctas, logits):
    """(logits 0: every key weighs the same; 20: some steps lie a hundred binades below others)"""
    for spread in (0, 3):
        a, b = batch(APART[case], d, len(case), spread, logits)
        check(a, b, ctas, d ** -0.5, spread)


@gpu
@pytest.mark.parametrize("d", [64, 128])
def test_many_keys_of_the_smallest_size(d):
    """30000 keys a stream with rows of 2^-110, most of them 7.75 binades heavier than the first."""
    nk, page = 60000, 64
    table, pool = table_for([nk], page, 0, 1)
    codes, exps = random_cache(pool, 1, page, d, 1)
    codes[1] &= 0xBF
    codes[0] = 0x38  # 1
    exps[0] = 127
    for j in range(2 * STEP):
        codes[0][int(table[0, j // page]), :, j % page] = 0
    exps[1] = 127 - 110
    scale = 7.75 * float(np.log(2.0)) / d
    q, mask = torch.ones(2, 1, d).bfloat16(), words_of(ancestors([-1, 0]), 1)
    check((q, codes, exps, mask, 2, nk, table), (codes, exps, page), 1, scale)


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


@gpu
@pytest.mark.parametrize("ctas", [1, 3])
@pytest.mark.parametrize("pattern", [[-110, 120], [120, -110], [-110, -110, 120, 120]])
def test_nan_codes_of_small_rows_next_to_large_ones(pattern, ctas):
    """A NaN code of a key that every token sees reaches every token, whatever its row's size."""
    a, _ = batch(pattern, 128, 5)
    codes, exps, table = a[1], a[2], a[6]
    j = STEP * pattern.index(-110) + 7
    codes[1][int(table[0, j // 64]), :, j % 64, 11] = 0x7F
    o, lse = run(a, ctas, 0.1)
    nan = torch.isnan(o)
    assert nan[..., 11].all() and nan.sum() == nan[..., 11].numel() and torch.isfinite(lse).all()


@gpu
@pytest.mark.parametrize("d", [64, 128])
def test_the_sum_does_not_depend_on_the_values(d):
    """lse is the cache decode's, whatever lies in V."""
    for pattern in ([118], [120, -110], [ZERO, 40], [-110]):
        a, _ = batch(pattern, d, 2, H=2)
        q, codes, exps, _, nq, nk, table = a
        chain = fa.tree_mask(ints(range(-1, nq - 1)).cuda(), cu([nq]).cuda(), nq).cpu()
        got = run((q, codes, exps, chain, nq, nk, table), 2, 0.1)[1]
        want = fa.forward_decode_cache(q.cuda(), to_cache(codes, exps), cu([nq]).cuda(), ints([nk]).cuda(), table.cuda(),
                                       nq, nk, 0.1, True)[1]
        assert (got - want).abs().max() < 2e-5, pattern


@gpu
@pytest.mark.parametrize("ctas", [1, 3])
@pytest.mark.parametrize("e", [-90, 0, 86])
@pytest.mark.parametrize("d", [64, 128])
def test_rows_of_zeros_that_weigh_the_most(d, e, ctas):
    """Keys 2^50 times the others' weight whose value rows are zeros lie among the others: those keep their bits."""
    nk, nq, page = 500, 4, 32
    table, pool = table_for([nk], page, 0, 1)
    codes, exps = random_cache(pool, 1, page, d, 1)
    codes[1] &= 0xBF
    exps[0], exps[1] = 121, 127 + e
    zero = np.random.RandomState(2).rand(*exps[1].shape) < 0.2
    codes[0][zero], exps[0][zero], codes[1][zero], exps[1][zero] = 0x38, 127, 0, 127
    plain = exps.copy()
    plain[1][zero] = 1
    q, mask = torch.ones(nq, 2, d).bfloat16(), words_of(ancestors([-1, 0, 0, 1]), 1)
    check((q, codes, exps, mask, nq, nk, table), (codes, plain, page), ctas, 50 * float(np.log(2.0)) / d)
