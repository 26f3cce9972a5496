"""Split-KV decode over the paged e4m3 cache (fa_fwd_decode_cache) against attention in 64 bits on
the cached values: head layouts, head sizes, page sizes, lengths from zero on, masks that leave
rows empty, thread block counts; what lies behind a sequence's end and in missing pages; NaN codes that
only some queries see; rows far apart in size; padded batches, streams, graphs, determinism;
refusals."""
import ctypes

import numpy as np
import pytest
import torch

import exact_attention_25_gb300 as fa
from tests.gpu_util import guarded_empty
from tests.serve_util import attention_rows, check_rows, values
from tests.test_cache import cu, table_for

gpu = pytest.mark.gpu
F16_STEP = 2.0 ** -11  # the softmax weights are rounded to f16


def random_cache(pool, Hkv, page, d, seed, spread=2):
    """Codes drawn over all finite ones, exponents around 2^-7 (values of order 1)."""
    r = np.random.RandomState(seed)
    codes = r.randint(0, 256, (2, pool, Hkv, page, d)).astype(np.uint8)
    codes[codes & 127 == 127] = 0x70
    exps = (120 + r.randint(-spread, spread + 1, (2, pool, Hkv, page))).astype(np.uint8)
    return codes, exps


def to_cache(codes, exps):
    t = [torch.tensor(x).cuda() for x in (codes[0], codes[1], exps[0], exps[1])]
    return fa.PagedCache(*t)


def sequence(codes, exps, z, table, b, hk, n, page):
    """fp64 rows 0 .. n-1 of a sequence and head."""
    at = np.arange(n)
    p = table[b].numpy()[at // page]
    return values(codes[z][p, hk, at % page], exps[z][p, hk, at % page])


def row_scale(exps, table, b, hk, n, page):
    at = np.arange(n)
    return np.exp2(exps[table[b].numpy()[at // page], hk, at % page].astype(np.float64) - 127)


def reference(q, codes, exps, table, lens_q, lens_k, H, page, scale, causal, tok0=0):
    T, _, d = q.shape
    Hkv = codes.shape[2]
    ref = [np.zeros((T, H, d)), np.full((H, T), -np.inf), np.zeros((T, H, d)), np.zeros((H, T)),
           np.zeros((T, H, d))]
    t = tok0
    for b, (n, nk) in enumerate(zip(lens_q, lens_k)):
        for h in range(H):
            hk = h // (H // Hkv)
            k, v = (sequence(codes, exps, z, table, b, hk, nk, page) for z in (0, 1))
            o, lse, pv, mag, low = attention_rows(
                q[t:t + n, h].double().numpy(), k, v, scale, causal, nk - n,
                row_scale(exps[1], table, b, hk, nk, page))
            ref[0][t:t + n, h], ref[1][h, t:t + n] = o, lse
            ref[2][t:t + n, h], ref[3][h, t:t + n], ref[4][t:t + n, h] = pv, mag, low
        t += n
    return ref


def run_case(lens_q, lens_k, H, Hkv, d, page, causal, ctas, seed, scale=None, spread=2):
    table, pool = table_for(lens_k, page, 1, seed)
    codes, exps = random_cache(pool, Hkv, page, d, seed, spread)
    q = torch.randn(sum(lens_q), H, d, generator=torch.Generator().manual_seed(seed)).bfloat16()
    scale = d ** -0.5 if scale is None else scale
    got = fa.forward_decode_cache(
        q.cuda(), to_cache(codes, exps), cu(lens_q).cuda(),
        torch.tensor(lens_k, dtype=torch.int32).cuda(), table.cuda(), max(lens_q),
        max(max(lens_k), 1), scale, causal, ctas)
    fa.fa_device_status()
    ref = reference(q, codes, exps, table, lens_q, lens_k, H, page, scale, causal)
    return _check(got, ref)


def _check(got, ref, what=""):
    return check_rows(got[0].transpose(0, 1), got[1], ref[0].transpose(1, 0, 2), ref[1],
                      ref[2].transpose(1, 0, 2), ref[3], ref[4].transpose(1, 0, 2), F16_STEP, what)


CASES = {
    # name: (query lengths, key lengths, H, Hkv, page)
    "one_key": ([1], [1], 1, 1, 16),
    "one_token_mha": ([1, 1, 1], [1, 64, 500], 3, 3, 16),
    "gqa4": ([1, 1, 1, 1], [129, 128, 700, 15], 8, 2, 64),
    "gqa7": ([1, 2], [300, 65], 7, 1, 32),
    "mqa16": ([1, 1], [333, 64], 16, 1, 128),
    "speculative": ([4, 4, 2, 1], [300, 130, 2, 63], 8, 2, 64),
    "rows_17_to_32": ([3, 2], [200, 77], 16, 2, 16),
    "rows_33_to_64": ([7, 5], [200, 301], 8, 1, 64),
    "many_row_chunks": ([40, 11, 33], [90, 200, 20], 12, 2, 32),
    "empty_sequences": ([1, 0, 1, 1, 2], [0, 50, 260, 1, 0], 4, 2, 256),
    "more_queries_than_keys": ([5, 9, 1], [3, 8, 1], 4, 1, 16),
}


@gpu
@pytest.mark.parametrize("ctas", [None, 1, 2, 3, 7, 29])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("case", list(CASES))
def test_decode_cache_against_64_bits(case, d, causal, ctas):
    lens_q, lens_k, H, Hkv, page = CASES[case]
    worst = run_case(lens_q, lens_k, H, Hkv, d, page, causal, ctas, seed=7 * len(case) + d)
    print(case, d, causal, ctas, worst)


@gpu
@pytest.mark.parametrize("scale", [-0.2, 0.0, 1.5])
@pytest.mark.parametrize("d", [64, 128])
def test_decode_cache_scales(d, scale):
    run_case([1, 3], [200, 70], 4, 2, d, 64, True, 2, seed=5, scale=scale)


@gpu
@pytest.mark.parametrize("d", [64, 128])
def test_rows_of_very_different_size(d):
    """K and V rows whose scales lie up to 2^60 apart (the scores stay moderate: the large K rows
    are nearly orthogonal to the queries by their codes being zero elsewhere)."""
    H, Hkv, page, nk = 4, 2, 32, 150
    table, pool = table_for([nk], page, 1, 3)
    codes, exps = random_cache(pool, Hkv, page, d, 4)
    r = np.random.RandomState(1)
    exps[1] = (127 + r.randint(-30, 31, exps[1].shape)).astype(np.uint8)   # V: 2^-30 .. 2^30
    exps[0] = (127 + r.randint(-30, -6, exps[0].shape)).astype(np.uint8)   # K: tiny to moderate
    q = torch.randn(1, H, d, generator=torch.Generator().manual_seed(2)).bfloat16()
    q[0, 0] *= 2.0 ** -40   # query rows of any size, too
    q[0, 1] *= 2.0 ** 20
    got = fa.forward_decode_cache(q.cuda(), to_cache(codes, exps), cu([1]).cuda(),
                                  torch.tensor([nk], dtype=torch.int32).cuda(), table.cuda(), 1,
                                  nk, 2.0 ** -16, False, 3)
    ref = reference(q, codes, exps, table, [1], [nk], H, page, 2.0 ** -16, False)
    _check(got, ref)


@gpu
@pytest.mark.parametrize("ctas", [1, 3])
@pytest.mark.parametrize("d", [64, 128])
def test_a_peaked_row_keeps_its_long_tail(d, ctas):
    """One key far above the rest in weight and thousands of light ones: what the light ones add
    in the columns where the heavy one is zero is kept (weights are not flushed)."""
    H, Hkv, page, nk = 1, 1, 64, 4096
    table, pool = table_for([nk], page, 0, 1)
    codes = np.zeros((2, pool, Hkv, page, d), np.uint8)
    exps = np.full((2, pool, Hkv, page), 127, np.uint8)
    one = 0x38
    codes[0, ..., 0] = 0x38 | 0x80           # K = -1 in column 0: logit 0 relative to the peak's
    codes[1, ..., 1:] = one                  # V = 1 everywhere but column 0
    p, r = int(table[0, 5]), 9
    codes[0, p, 0, r, 0], codes[1, p, 0, r] = one, 0
    codes[1, p, 0, r, 0] = one
    q = torch.zeros(1, 1, d).bfloat16()
    q[0, 0, 0] = 8.0                         # logits +8 and -8: a weight of e^-16 each
    got = fa.forward_decode_cache(q.cuda(), to_cache(codes, exps), cu([1]).cuda(),
                                  torch.tensor([nk], dtype=torch.int32).cuda(), table.cuda(), 1,
                                  nk, 1.0, False, ctas)
    ref = reference(q, codes, exps, table, [1], [nk], H, page, 1.0, False)
    assert ref[0][0, 0, 1] > 1e-4
    _check(got, ref)


def poisoned(case_seed, lens_q, lens_k, H, Hkv, d, page):
    """A case whose pages hold NaN codes and wild exponents wherever no key lies."""
    table, pool = table_for(lens_k, page, 2, case_seed)
    codes, exps = random_cache(pool, Hkv, page, d, case_seed)
    used = np.zeros((pool, page), bool)
    for b, n in enumerate(lens_k):
        at = np.arange(n)
        used[table[b].numpy()[at // page], at % page] = True
    for z in range(2):
        codes[z][np.broadcast_to(~used[:, None], (pool, Hkv, page))] = 0x7F
        exps[z][np.broadcast_to(~used[:, None], (pool, Hkv, page))] = 255
    q = torch.randn(sum(lens_q), H, d, generator=torch.Generator().manual_seed(1)).bfloat16()
    return table, codes, exps, q


@gpu
@pytest.mark.parametrize("ctas", [1, 2])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [16, 64, 128])
def test_what_lies_behind_the_end_is_not_seen(page, d, causal, ctas):
    lens_q, lens_k, H, Hkv = [1, 3, 2], [70, 129, 1], 4, 2
    table, codes, exps, q = poisoned(6, lens_q, lens_k, H, Hkv, d, page)
    got = fa.forward_decode_cache(q.cuda(), to_cache(codes, exps), cu(lens_q).cuda(),
                                  torch.tensor(lens_k, dtype=torch.int32).cuda(), table.cuda(), 3,
                                  129, 0.1, causal, ctas)
    fa.fa_device_status()
    _check(got, reference(q, codes, exps, table, lens_q, lens_k, H, page, 0.1, causal))


@gpu
@pytest.mark.parametrize("what", ["k", "v", "k_exp", "v_exp"])
@pytest.mark.parametrize("d", [64, 128])
def test_nan_of_a_late_key_reaches_only_the_queries_that_see_it(d, what):
    lens_q, lens_k, H, Hkv, page = [12], [100], 4, 2, 16
    table, pool = table_for(lens_k, page, 1, 2)
    codes, exps = random_cache(pool, Hkv, page, d, 9)
    j = 93  # seen by queries 5 .. 11 (of 12, over keys 88 .. 99)
    p, r = int(table[0, j // page]), j % page
    z = 0 if what[0] == "k" else 1
    if what.endswith("exp"):
        exps[z][p, 1, r] = 255
    else:
        codes[z][p, 1, r, 5] = 0xFF
    vals = to_cache(codes, exps)
    q = torch.randn(12, H, d, generator=torch.Generator().manual_seed(3)).bfloat16()
    o, lse = fa.forward_decode_cache(q.cuda(), vals, cu(lens_q).cuda(),
                                     torch.tensor(lens_k, dtype=torch.int32).cuda(), table.cuda(),
                                     12, 100, 0.1, True, 2)
    nan = torch.isnan(o).cpu()
    want = torch.zeros_like(nan)
    heads = slice(2, 4)  # the group of key/value head 1
    if what == "v":
        want[5:, heads, 5] = True
    else:
        want[5:, heads] = True
    assert torch.equal(nan, want)
    if what[0] == "k":
        assert torch.isnan(lse[heads, 5:]).all()
    # the rest is what it was without the NaN
    if what.endswith("exp"):
        exps[z][p, 1, r] = 127
    else:
        codes[z][p, 1, r, 5] = 0
    ref = reference(q, codes, exps, table, lens_q, lens_k, H, page, 0.1, True)
    o = torch.where(nan.cuda(), torch.zeros_like(o), o)
    for x in (ref[0], ref[2], ref[4]):
        x[nan.numpy()] = 0.0
    if what[0] == "k":
        lse = lse.clone()
        lse[heads, 5:] = torch.tensor(ref[1][heads, 5:]).float().cuda()
    _check((o, lse), ref)


@gpu
@pytest.mark.parametrize("ctas", [1, 3])
def test_missing_pages_are_left_out(ctas):
    """Table entries outside the pool: their keys take no part, whatever the mask."""
    H, Hkv, d, page, nk = 4, 1, 128, 16, 200
    table, pool = table_for([nk], page, 0, 4)
    codes, exps = random_cache(pool, Hkv, page, d, 3)
    q = torch.randn(1, H, d, generator=torch.Generator().manual_seed(4)).bfloat16()
    holes = table.clone()
    for i, bad in ((0, -1), (5, pool), (6, 2 ** 31 - 1), (12, -2 ** 31)):
        holes[0, i] = bad
    got = fa.forward_decode_cache(q.cuda(), to_cache(codes, exps), cu([1]).cuda(),
                                  torch.tensor([nk], dtype=torch.int32).cuda(), holes.cuda(), 1,
                                  nk, 0.1, False, ctas)
    fa.fa_device_status()
    keep = np.array([j for j in range(nk) if j // page not in (0, 5, 6, 12)])
    for h in range(H):
        k, v = (sequence(codes, exps, z, table, 0, 0, nk, page)[keep] for z in (0, 1))
        s = row_scale(exps[1], table, 0, 0, nk, page)[keep]
        check_rows(got[0][:, h], got[1][h],
                   *attention_rows(q[:, h].double().numpy(), k, v, 0.1, False, 0, s), F16_STEP)


@gpu
@pytest.mark.parametrize("ctas", [1, 4])
def test_padded_batches_guards_and_repeats(ctas):
    """Tokens before the first and behind the last sequence stay as they are, nothing outside the
    outputs and the workspace is written, and a second call gives the same bits."""
    lens_q, lens_k, H, Hkv, d, page = [2, 0, 1], [130, 9, 64], 6, 2, 64, 32
    pad0, pad1 = 3, 5
    table, pool = table_for(lens_k, page, 1, 8)
    codes, exps = random_cache(pool, Hkv, page, d, 8)
    T = pad0 + sum(lens_q) + pad1
    q = torch.randn(T, H, d, generator=torch.Generator().manual_seed(5)).bfloat16()
    starts = (cu(lens_q) + pad0).to(torch.int32).cuda()
    n = torch.tensor(lens_k, dtype=torch.int32).cuda()
    cache = to_cache(codes, exps)
    outs = []
    for _ in range(2):
        o, ow = guarded_empty((T, H, d), torch.bfloat16)
        lse, lw = guarded_empty((H, T), torch.float32)
        o.fill_(3.0)
        lse.fill_(4.0)
        nbytes = fa.fa_decode_cache_workspace_bytes(H, Hkv, d, 2, ctas)
        ws, ww = guarded_empty((max(nbytes, 16),), torch.uint8)
        ws.fill_(0xFF)  # NaNs
        fa.fa_fwd_decode_cache(q.cuda(), cache, o, lse, starts, n, table.cuda(), 2, 130, 0.1, True,
                               ctas, ws if nbytes else None)
        fa.fa_device_status()
        for w in (ow, lw, ww):
            w()
        outs.append((o.clone(), lse.clone()))
    o, lse = outs[0]
    assert torch.equal(o, outs[1][0]) and torch.equal(lse, outs[1][1])
    for part in (slice(0, pad0), slice(T - pad1, T)):
        assert (o[part] == 3.0).all() and (lse[:, part] == 4.0).all()
    ref = reference(q, codes, exps, table, lens_q, lens_k, H, page, 0.1, True, tok0=pad0)
    mid = slice(pad0, T - pad1)
    _check((o[mid], lse[:, mid]), [x[mid] if i % 2 == 0 else x[:, mid] for i, x in enumerate(ref)])


@gpu
def test_malformed_lengths_stay_inside():
    """Starts that do not rise, lengths past the table and negative ones: values without meaning,
    but no access outside the tensors and no failure."""
    H, Hkv, d, page, pool = 4, 2, 64, 16, 5
    codes, exps = random_cache(pool, Hkv, page, d, 1)
    cache = to_cache(codes, exps)
    table = torch.randint(0, pool, (3, 2), dtype=torch.int32).cuda()
    q = torch.randn(6, H, d).bfloat16().cuda()
    for starts, lens in (([0, 5, 2, 6], [900, -3, 32]), ([-4, 2, 9, 3], [2 ** 31 - 1, 0, 31]),
                         ([6, 6, 0, 100], [-2 ** 31, 33, 64])):
        o, ow = guarded_empty((6, H, d), torch.bfloat16)
        lse, lw = guarded_empty((H, 6), torch.float32)
        ws = torch.empty(fa.fa_decode_cache_workspace_bytes(H, Hkv, d, 6, 3), dtype=torch.uint8).cuda()
        fa.fa_fwd_decode_cache(q, cache, o, lse, torch.tensor(starts, dtype=torch.int32).cuda(),
                               torch.tensor(lens, dtype=torch.int32).cuda(), table, 6, 1000, 0.1,
                               True, 3, ws)
        fa.fa_device_status()
        ow()
        lw()


@gpu
def test_decode_cache_streams_and_graphs():
    """A step captured with its append: replays follow the cache as it grows; two graphs with
    workspaces of their own run on two streams at once; a call on another stream."""
    H, Hkv, d, page, B = 8, 2, 128, 64, 2
    lens = [100, 63]
    table, pool = table_for([n + 16 for n in lens], page, 1, 2)
    codes, exps = random_cache(pool, Hkv, page, d, 2)
    cache, tab, ones = to_cache(codes, exps), table.cuda(), cu([1] * B).cuda()
    most = max(lens) + 16

    def make():
        n = torch.tensor(lens, dtype=torch.int32).cuda()
        mine = fa.PagedCache(*(t.clone() for t in cache))
        q, k, v = (torch.randn(B, h, d).bfloat16().cuda() for h in (H, Hkv, Hkv))
        o, lse = torch.empty_like(q), torch.empty(H, B, device="cuda")
        ws = torch.empty(fa.fa_decode_cache_workspace_bytes(H, Hkv, d, 1, 2), dtype=torch.uint8).cuda()

        def step():
            n.add_(1)
            fa.cache_append(mine, k, v, ones, n, tab, 1)
            fa.fa_fwd_decode_cache(q, mine, o, lse, ones, n, tab, 1, most, 0.1, True, 2, ws)

        return n, mine, q, k, v, o, lse, step

    states = [make(), make()]
    for s in states:  # a first call outside capture, then undo its step
        s[-1]()
        s[0].sub_(1)
    graphs = []
    for s in states:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            s[-1]()
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(8):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for n, mine, q, k, v, o, lse, _ in states:
        assert n.tolist() == [x + 8 for x in lens]
        want = fa.forward_decode_cache(q, mine, ones, n, tab, 1, most, 0.1, True, 2)
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        got = fa.forward_decode_cache(q, mine, ones, n, tab, 1, most, 0.1, True, 2, stream=side)
        side.synchronize()
        assert torch.equal(got[0], want[0])
    fa.fa_device_status()


@gpu
def test_decode_cache_at_serving_size():
    """8 sequences of up to 9000 keys, 32 heads over 8, the suggested split count; every head of
    two groups."""
    lens_k, H, Hkv, d, page = [9000, 1, 4097, 8191, 777, 64, 2050, 6000], 32, 8, 128, 64
    table, pool = table_for(lens_k, page, 3, 1)
    codes, exps = random_cache(pool, Hkv, page, d, 1)
    q = torch.randn(8, H, d, generator=torch.Generator().manual_seed(0)).bfloat16()
    o, lse = fa.forward_decode_cache(q.cuda(), to_cache(codes, exps), cu([1] * 8).cuda(),
                                     torch.tensor(lens_k, dtype=torch.int32).cuda(), table.cuda(),
                                     1, 9000, None, True)
    fa.fa_device_status()
    heads = [4, 5, 6, 7, 24, 25, 26, 27]
    ref = reference(q[:, heads], codes[:, :, [1, 6]], exps[:, :, [1, 6]], table, [1] * 8, lens_k, 8,
                    page, d ** -0.5, True)
    _check((o[:, heads], lse[heads]), ref)


# ------------------------------------------------------------------------------ refusals (CPU)

@pytest.fixture(scope="module")
def lib():
    from exact_attention_25_gb300 import _lib, build

    build.build()
    return _lib.load(_lib.LIB_PATH)


@pytest.mark.parametrize("kw, code", [
    (dict(d=96), -2), (dict(B=0), -1), (dict(Hkv=0), -1), (dict(H=3), -1), (dict(H=0), -1),
    (dict(total=0), -1), (dict(mq=0), -1), (dict(mk=0), -1), (dict(causal=2), -1),
    (dict(scale=float("nan")), -1), (dict(scale=float("inf")), -1), (dict(ctas=0), -1),
    (dict(ctas=4097), -1), (dict(page=24), -1), (dict(pages=0), -1), (dict(max_pages=0), -1),
    (dict(q=0), -1), (dict(o=0), -1), (dict(kc=0), -1), (dict(ke=0), -1), (dict(cu=0), -1),
    (dict(n=0), -1), (dict(table=0), -1), (dict(q=0x10008), -3), (dict(vc=0x40008), -3),
    (dict(lse=0x80002), -3), (dict(n=0x92001), -3), (dict(ws=0), -4), (dict(wsb=64), -4),
    (dict(ws=0xA0004), -3), (dict(pages=1 << 26, page=32), -7),
    (dict(total=1 << 25, H=4, mq=1), -7),
    (dict(B=1 << 28, mq=64, total=64, mk=1 << 20, max_pages=1 << 16), -7),
])
def test_decode_cache_refuses(lib, kw, code):
    a = dict(q=0x10000, kc=0x30000, vc=0x40000, ke=0x50000, ve=0x60000, o=0x70000, lse=0x80000,
             cu=0x91000, n=0x92000, table=0x93000, B=1, mq=1, mk=100, total=1, max_pages=8, pages=8,
             page=16, H=4, Hkv=2, d=64, scale=0.1, causal=0, ctas=2, ws=0xA0000, wsb=1 << 20)
    a.update(kw)
    vp = ctypes.c_void_p
    rc = lib.fa_fwd_decode_cache(
        vp(a["q"]), vp(a["kc"]), vp(a["vc"]), vp(a["ke"]), vp(a["ve"]), vp(a["o"]), vp(a["lse"]),
        vp(a["cu"]), vp(a["n"]), vp(a["table"]), a["B"], a["mq"], a["mk"], a["total"],
        a["max_pages"], a["pages"], a["page"], a["H"], a["Hkv"], a["d"], ctypes.c_float(a["scale"]),
        a["causal"], a["ctas"], vp(a["ws"]), a["wsb"], None)
    assert rc == code


def test_thread_block_rule(lib):
    f, w = lib.fa_decode_cache_ctas_for, lib.fa_decode_cache_workspace_bytes
    assert f(1, 8, 8, 1, 1, 152) == 4                       # one for every two blocks of keys
    assert f(1, 32, 8, 1, 4096, 152) == 8 * 32 / 2
    assert f(8, 32, 8, 1, 32768, 152) == 304
    assert f(1, 64, 1, 3, 100, 152) == 2                    # 192 query rows: three sets of 64
    assert f(0, 8, 8, 1, 1, 152) == -1 and f(1, 9, 8, 1, 1, 152) == -1 and f(1, 8, 8, 1, 1, 0) == -1
    assert w(8, 2, 64, 1, 1) == 0 and w(8, 2, 96, 1, 2) == 0 and w(8, 2, 64, 1, 4097) == 0
    for mq, rows in ((1, 8), (3, 16), (5, 32), (9, 64), (100, 64)):   # of 4 heads a group
        n = w(8, 2, 64, mq, 10)
        assert 20 * rows * 65 * 4 <= n <= 20 * rows * 65 * 4 + 3 * 256
