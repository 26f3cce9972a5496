"""Cached value rows of zeros add nothing to an output, and must not cost the other rows bits: the decode's f16
weights are framed by the largest product of a weight and its row's scale, and a row of zeros is kept under
scale 1, far above the rows of a head whose values are small.  Against attention in 64 bits, with a bound on the
weights' last bits that only rows with nonzero codes enter."""
import numpy as np
import pytest
import torch

import exact_attention_25_gb300 as fa
from tests.serve_util import attention_rows, check_rows
from tests.test_cache import cu, table_for
from tests.test_decode_cache import F16_STEP, random_cache, row_scale, sequence, to_cache

gpu = pytest.mark.gpu


def reference(q, codes, exps, table, lens_q, lens_k, H, page, scale, causal):
    T, _, d = q.shape
    Hkv = codes.shape[2]
    out = [np.zeros((H, T, d)), np.full((H, T), -np.inf), np.zeros((H, T, d)), np.zeros((H, T)), np.zeros((H, T, d))]
    t = 0
    for b, (n, nk) in enumerate(zip(lens_q, lens_k)):
        for h in range(H):
            hk = h // (H // Hkv)
            k, v = (sequence(codes, exps, z, table, b, hk, nk, page) for z in (0, 1))
            s = np.where((v != 0).any(-1), row_scale(exps[1], table, b, hk, nk, page), 2.0 ** -300)
            for x, y in zip(out, attention_rows(q[t:t + n, h].double().numpy(), k, v, scale, causal, nk - n, s)):
                x[h, t:t + n] = y
        t += n
    return out


def check(got, ref):
    return check_rows(got[0].transpose(0, 1), got[1], *ref, F16_STEP)


@gpu
@pytest.mark.parametrize("ctas", [1, 5])
@pytest.mark.parametrize("lens_q, H, Hkv", [([1, 1], 4, 2), ([4, 3], 8, 2), ([9, 2], 4, 1)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("size", [-24, -40, -90])
def test_zero_rows_cost_small_rows_nothing(size, d, lens_q, H, Hkv, ctas):
    page, lens_k = 32, [700, 150]
    table, pool = table_for(lens_k, page, 1, 5)
    codes, exps = random_cache(pool, Hkv, page, d, 3)
    exps[1] = (127 + size + np.random.RandomState(1).randint(-2, 3, exps[1].shape)).astype(np.uint8)
    for b, zeros in enumerate(([0, 5, 17, 130, 131, 400, 699], [3, 149])):
        for i, j in enumerate(zeros):
            p, r = int(table[b, j // page]), j % page
            codes[1, p, :, r] = 0x80 if i % 2 else 0   # zeros of both signs
            exps[1, p, :, r] = 127
    q = torch.randn(sum(lens_q), H, d, generator=torch.Generator().manual_seed(d)).bfloat16()
    for causal in (False, True):
        got = fa.forward_decode_cache(q.cuda(), to_cache(codes, exps), cu(lens_q).cuda(),
                                      torch.tensor(lens_k, dtype=torch.int32).cuda(), table.cuda(), max(lens_q),
                                      700, d ** -0.5, causal, ctas)
        fa.fa_device_status()
        check(got, reference(q, codes, exps, table, lens_q, lens_k, H, page, d ** -0.5, causal))


@gpu
@pytest.mark.parametrize("d", [64, 128])
def test_sequences_of_zero_rows(d):
    """Only rows of zeros: O = 0 under the scores' own lse; and rows that reach 448 beside them, kept under the
    same scale, count as ever."""
    H, Hkv, page, lens_k = 4, 2, 16, [200, 77, 300]
    table, pool = table_for(lens_k, page, 0, 6)
    codes, exps = random_cache(pool, Hkv, page, d, 4)
    zero = np.zeros((pool, page), bool)
    for b, every in ((0, 1), (1, 1), (2, 2)):
        at = np.arange(0, lens_k[b], every)
        zero[table[b].numpy()[at // page], at % page] = True
    codes[1][np.broadcast_to(zero[:, None], (pool, Hkv, page))] = 0
    exps[1][:] = 127
    q = torch.randn(3, H, d, generator=torch.Generator().manual_seed(2)).bfloat16()
    got = fa.forward_decode_cache(q.cuda(), to_cache(codes, exps), cu([1] * 3).cuda(),
                                  torch.tensor(lens_k, dtype=torch.int32).cuda(), table.cuda(), 1, 300, 0.1, True, 3)
    fa.fa_device_status()
    assert (got[0][:2] == 0).all() and torch.isfinite(got[1]).all()
    check(got, reference(q, codes, exps, table, [1] * 3, lens_k, H, page, 0.1, True))


@gpu
@pytest.mark.parametrize("d", [64, 128])
def test_appended_zero_rows_beside_small_values(d):
    """Through the calls that a user makes: padding tokens whose values are zero go into the cache."""
    H, Hkv, page, n = 8, 2, 64, 512
    g = torch.Generator().manual_seed(d)
    k, v, q = (torch.randn(m, h, d, generator=g).bfloat16() for m, h in ((n, Hkv), (n, Hkv), (1, H)))
    v = (v.float() * 2.0 ** -26).bfloat16()
    v[[0, 100, 511]] = 0.0
    table, pool = table_for([n], page, 1, 2)
    cache, lens = fa.new_cache(pool, page, Hkv, d), torch.tensor([n], dtype=torch.int32).cuda()
    fa.cache_append(cache, k.cuda(), v.cuda(), cu([n]).cuda(), lens, table.cuda(), n)
    got = fa.forward_decode_cache(q.cuda(), cache, cu([1]).cuda(), lens, table.cuda(), 1, n, causal=True)
    fa.fa_device_status()
    host = [t.view(torch.uint8).cpu().numpy() for t in cache]
    check(got, reference(q, np.stack(host[:2]), np.stack(host[2:]), table, [1], [n], H, page, d ** -0.5, True))
