"""Decoding with shared prefixes (fa_fwd_decode_shared) against attention in 64 bits over prefix and
own keys together: groups, head layouts, head sizes, lengths from zero on, thread block counts; what
lies behind the sequences; infinities and NaNs that only some queries see; padded batches, streams,
graphs, determinism; agreement with the plain decode, and with the cache; refusals."""
import ctypes

import numpy as np
import pytest
import torch

import exact_attention_25_gb300 as fa
from tests.gpu_util import guarded_empty
from tests.serve_util import attention_rows, check_rows
from tests.test_cache import cu, table_for

gpu = pytest.mark.gpu
# the softmax weights are rounded to bf16 (half a step: 2^-8), in the products and in the sum that
# divides them: each side moves O by at most that times sum p|v|
BF16_STEP = 2.0 ** -7


def make(lens_q, lens_k, group, prefix, H, Hkv, d, seed, pad=(0, 0), behind=None):
    """pad: query rows before the first and behind the last sequence; behind: value of 40 key rows
    behind the sequences' and the prefixes'."""
    g = torch.Generator().manual_seed(seed)
    rnd = lambda n, h: torch.randn(n, h, d, generator=g).bfloat16()  # noqa: E731
    x = dict(q=rnd(sum(lens_q) + sum(pad), H))
    for name, n in (("k", sum(lens_k)), ("v", sum(lens_k)), ("kp", sum(prefix)), ("vp", sum(prefix))):
        x[name] = rnd(n, Hkv)
        if behind is not None or n == 0:
            x[name] = torch.cat([x[name], torch.full((40, Hkv, d), behind or 0.0).bfloat16()])
    x.update(cu_q=cu(lens_q) + pad[0], cu_k=cu(lens_k), cu_g=torch.tensor(group, dtype=torch.int32),
             cu_p=cu(prefix))
    x["sizes"] = (max(max(lens_q), 1), max(max(lens_k), 1),
                  max([sum(lens_q[a:b]) for a, b in zip(group, group[1:])] + [1]), max(max(prefix), 1))
    return {n: t.to(torch.int32) if n.startswith("cu") else t for n, t in x.items()}


def run(x, scale, causal, ctas=None, stream=None):
    dev = {n: t.cuda() for n, t in x.items() if n != "sizes"}
    return fa.forward_decode_shared(dev["q"], dev["kp"], dev["vp"], dev["k"], dev["v"], dev["cu_q"],
                                    dev["cu_k"], dev["cu_g"], dev["cu_p"], *x["sizes"], scale,
                                    causal, ctas, stream)


def reference(x, scale, causal):
    q = x["q"].double().numpy()
    T, H, d = q.shape
    Hkv = x["k"].shape[1]
    ref = [np.zeros((T, H, d)), np.full((H, T), -np.inf), np.zeros((T, H, d)), np.zeros((H, T)),
           np.zeros((T, H, d))]
    cq, ck, cg, cp = (x[n].tolist() for n in ("cu_q", "cu_k", "cu_g", "cu_p"))
    for b in range(len(cq) - 1):
        g = next((g for g in range(len(cg) - 1) if cg[g] <= b < cg[g + 1]), None)
        p0, p1 = (cp[g], cp[g + 1]) if g is not None else (0, 0)
        n, nk = cq[b + 1] - cq[b], ck[b + 1] - ck[b]
        at = slice(cq[b], cq[b + 1])
        for h in range(H):
            hk = h // (H // Hkv)
            k, v = (torch.cat([x[a][p0:p1, hk], x[c][ck[b]:ck[b + 1], hk]]).double().numpy()
                    for a, c in (("kp", "k"), ("vp", "v")))
            o, lse, pv, mag, low = attention_rows(q[at, h], k, v, scale, causal, p1 - p0 + nk - n,
                                                  always=p1 - p0)
            ref[0][at, h], ref[1][h, at], ref[2][at, h], ref[3][h, at] = o, lse, pv, mag
    return ref


def check(got, ref, what=""):
    return check_rows(got[0].transpose(0, 1), got[1], ref[0].transpose(1, 0, 2), ref[1],
                      ref[2].transpose(1, 0, 2), ref[3], ref[4].transpose(1, 0, 2), BF16_STEP, what)


CASES = {
    # name: (query lengths, own key lengths, groups' first sequences, prefix lengths, H, Hkv)
    "one_token": ([1], [1], [0, 1], [1], 1, 1),
    "one_group": ([1, 1, 1, 1], [5, 128, 1, 300], [0, 4], [700], 8, 2),
    "three_groups": ([1, 2, 1, 1, 3], [7, 129, 64, 1, 3], [0, 2, 3, 5], [256, 1, 333], 4, 4),
    "gqa7": ([1, 1, 2], [30, 200, 2], [0, 3], [129], 7, 1),
    "gqa16_many_tiles": ([4] * 12, [9] * 12, [0, 12], [400], 32, 2),
    "mha_many_tokens": ([40, 1, 90], [40, 10, 90], [0, 3], [260], 2, 2),
    "group_of_128_heads": ([1, 2], [12, 140], [0, 2], [150], 128, 1),
    "nothing_of_some": ([1, 0, 2, 1, 1], [0, 9, 0, 4, 0], [0, 2, 2, 5], [0, 50, 0], 4, 2),
    "no_own_keys": ([1, 1], [0, 0], [0, 2], [100], 4, 1),
    "no_prefix": ([1, 3], [130, 40], [0, 2], [0], 4, 2),
    "outside_the_groups": ([1, 1, 1, 1], [20, 30, 0, 50], [1, 2], [90], 4, 2),
    "more_queries_than_keys": ([6, 3], [2, 1], [0, 1, 2], [20, 0], 4, 2),
    "long": ([1, 1, 1], [1000, 3, 257], [0, 3], [3000], 8, 2),
}


@gpu
@pytest.mark.parametrize("ctas", [None, 1, 5, 40])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("case", list(CASES))
def test_decode_shared_against_64_bits(case, d, causal, ctas):
    lens_q, lens_k, group, prefix, H, Hkv = CASES[case]
    x = make(lens_q, lens_k, group, prefix, H, Hkv, d, seed=len(case) + d)
    got = run(x, d ** -0.5, causal, ctas)
    fa.fa_device_status()
    print(case, d, causal, ctas, check(got, reference(x, d ** -0.5, causal)))


@gpu
@pytest.mark.parametrize("scale", [-0.2, 0.0, 1.0])
@pytest.mark.parametrize("d", [64, 128])
def test_decode_shared_scales(d, scale):
    x = make([2, 1], [150, 3], [0, 2], [200], 4, 2, d, 3)
    check(run(x, scale, True, 7), reference(x, scale, True))


@gpu
@pytest.mark.parametrize("what", [float("nan"), float("inf"), -3.0e38])
@pytest.mark.parametrize("d", [64, 128])
def test_what_lies_behind_the_sequences_is_not_seen(d, what):
    x = make([1, 3, 1], [70, 129, 1], [0, 3], [257], 4, 2, d, 5, behind=what)
    got = run(x, 0.1, True)
    fa.fa_device_status()
    check(got, reference(x, 0.1, True))
    x = make([2, 2], [0, 5], [0, 1, 2], [100, 30], 4, 2, d, 6, behind=what)
    check(run(x, 0.1, False, 4), reference(x, 0.1, False))


@gpu
@pytest.mark.parametrize("ctas", [None, 3])
@pytest.mark.parametrize("d", [64, 128])
def test_odd_values_of_a_late_key_reach_only_the_queries_that_see_it(d, ctas):
    """NaN and infinities in V at own keys that the later queries of a sequence see."""
    nq, nk = 10, 140
    x = make([1, nq], [30, nk], [0, 2], [90], 4, 2, d, 7)
    at = {133: (float("nan"), 3), 136: (float("inf"), 4), 138: (float("-inf"), 5)}
    for j, (val, c) in at.items():
        x["v"][30 + j, 1, c] = val
    o, lse = run(x, 0.1, True, ctas)
    fa.fa_device_status()
    o = o.cpu()
    clean = {n: t.clone() if torch.is_tensor(t) else t for n, t in x.items()}
    for j, (val, c) in at.items():
        clean["v"][30 + j, 1, c] = 0.0
    ref = reference(clean, 0.1, True)
    for j, (val, c) in at.items():
        first = j - (nk - nq)  # the first query of the sequence that sees key j
        hit = o[1 + first:, 2:4, c]
        assert torch.isnan(hit).all() if np.isnan(val) else (hit == val).all()
        o[1 + first:, 2:4, c] = 0.0
        for z in (0, 2):
            ref[z][1 + first:, 2:4, c] = 0.0
    check((o, lse), ref)


@gpu
def test_nan_of_a_prefix_reaches_its_group_only():
    x = make([1, 1, 1], [10, 10, 10], [0, 1, 3], [40, 50], 4, 2, 64, 8)
    x["kp"][5, 0, 0] = float("nan")          # group 0, key/value head 0
    x["vp"][60, 1, 7] = float("inf")         # group 1, head 1
    o, lse = run(x, 0.1, True)
    assert torch.isnan(o[0, :2]).all() and torch.isnan(lse[:2, 0]).all()
    assert torch.isfinite(o[0, 2:]).all() and torch.isfinite(o[1:, :2]).all()
    assert (o[1:, 2:, 7] == float("inf")).all() and torch.isfinite(lse[:, 1:]).all()


@gpu
@pytest.mark.parametrize("ctas", [1, 6])
def test_padded_batches_guards_and_repeats(ctas):
    pad = (3, 6)
    H, Hkv, d = 6, 2, 64
    x = make([2, 0, 1], [130, 9, 64], [0, 1, 3], [200, 77], H, Hkv, d, 9, pad=pad)
    T = x["q"].shape[0]
    dev = {n: t.cuda() for n, t in x.items() if n != "sizes"}
    outs = []
    for _ in range(2):
        o, ow = guarded_empty((T, H, d), torch.bfloat16)
        lse, lw = guarded_empty((H, T), torch.float32)
        o.fill_(3.0)
        lse.fill_(4.0)
        ws, ww = guarded_empty((fa.fa_decode_shared_workspace_bytes(T, H, d, ctas),), torch.uint8)
        ws.fill_(0xFF)  # NaNs
        fa.fa_fwd_decode_shared(dev["q"], dev["kp"], dev["vp"], dev["k"], dev["v"], o, lse,
                                dev["cu_q"], dev["cu_k"], dev["cu_g"], dev["cu_p"], *x["sizes"], 0.1,
                                True, ctas, ws)
        fa.fa_device_status()
        for w in (ow, lw, ww):
            w()
        outs.append((o.clone(), lse.clone()))
    o, lse = outs[0]
    assert torch.equal(o, outs[1][0]) and torch.equal(lse, outs[1][1])
    for part in (slice(0, pad[0]), slice(T - pad[1], T)):
        assert (o[part] == 3.0).all() and (lse[:, part] == 4.0).all()
    mid = slice(pad[0], T - pad[1])
    ref = reference(x, 0.1, True)
    check((o[mid], lse[:, mid]), [t[mid] if z % 2 == 0 else t[:, mid] for z, t in enumerate(ref)])


@gpu
def test_malformed_starts_stay_inside():
    H, Hkv, d, T = 4, 2, 64, 8
    q = torch.randn(T, H, d).bfloat16().cuda()
    k, kp = (torch.randn(50, Hkv, d).bfloat16().cuda() for _ in range(2))
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32).cuda()  # noqa: E731
    for cq, ck, cg, cp in (((0, 5, 2, 8), (0, 60, -3, 50), (0, 3), (0, 900)),
                           ((-4, 2, 9, 3), (50, 0, 20, 10), (2, 1), (30, 10)),
                           ((8, 8, 0, 100), (0, 9, 9, 2 ** 31 - 1), (-5, 77), (-2 ** 31, 2 ** 31 - 1))):
        o, ow = guarded_empty((T, H, d), torch.bfloat16)
        lse, lw = guarded_empty((H, T), torch.float32)
        ws, ww = guarded_empty((fa.fa_decode_shared_workspace_bytes(T, H, d, 9),), torch.uint8)
        fa.fa_fwd_decode_shared(q, kp, kp, k, k, o, lse, i32(*cq), i32(*ck), i32(*cg), i32(*cp), 8, 50,
                                8, 50, 0.1, True, 9, ws)
        fa.fa_device_status()
        ow()
        lw()
        ww()


@gpu
def test_agrees_with_the_plain_decode_of_repeated_prefixes():
    """The same batch with the prefix copied in front of every sequence's keys, through
    fa_fwd_decode: both within bf16 rounding of each other."""
    lens_q, lens_k, prefix, H, Hkv, d = [1, 3, 1], [40, 77, 129], 1000, 32, 8, 128
    x = make(lens_q, lens_k, [0, 3], [prefix], H, Hkv, d, 10)
    o, lse = run(x, None, True)
    at = np.cumsum([0] + lens_k)
    k, v = (torch.cat([t for b in range(3) for t in (x[a], x[c][at[b]:at[b + 1]])])
            for a, c in (("kp", "k"), ("vp", "v")))
    want = fa.forward_decode(x["q"].cuda(), k.cuda(), v.cuda(), x["cu_q"].cuda(),
                             cu([prefix + n for n in lens_k]).cuda(), 3, prefix + 129, causal=True)
    assert (o.float() - want[0].float()).abs().max().item() <= 1.6e-2
    assert (lse - want[1]).abs().max().item() <= 1e-3


@gpu
def test_streams_and_graphs():
    xs = [make([1, 1, 2], [40, 7, 300], [0, 3], [500], 8, 2, 128, s) for s in (1, 2)]
    want = [run(x, 0.1, True, 20) for x in xs]
    graphs, outs = [], []
    for x in xs:
        dev = {n: t.cuda() for n, t in x.items() if n != "sizes"}
        o, lse = torch.empty_like(dev["q"]), torch.empty(8, 4, device="cuda")
        ws = torch.empty(fa.fa_decode_shared_workspace_bytes(4, 8, 128, 20), dtype=torch.uint8).cuda()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            fa.fa_fwd_decode_shared(dev["q"], dev["kp"], dev["vp"], dev["k"], dev["v"], o, lse,
                                    dev["cu_q"], dev["cu_k"], dev["cu_g"], dev["cu_p"], *x["sizes"],
                                    0.1, True, 20, ws)
        graphs.append(g)
        outs.append((o, lse, dev, ws))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(4):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for (o, lse, _, _), w in zip(outs, want):
        assert torch.equal(o, w[0]) and torch.equal(lse, w[1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = run(xs[0], 0.1, True, 20, stream=side)
    side.synchronize()
    assert torch.equal(got[0], want[0][0])
    fa.fa_device_status()


@gpu
def test_at_serving_size():
    """24 continuations of two prompts, 32 heads over 8; every head of two groups."""
    r = np.random.RandomState(0)
    lens_k = r.randint(1, 600, 24).tolist()
    x = make([1] * 24, lens_k, [0, 10, 24], [4000, 2500], 32, 8, 128, 11)
    o, lse = run(x, None, True)
    fa.fa_device_status()
    heads, kv = [4, 5, 6, 7, 28, 29, 30, 31], [1, 7]
    part = dict(x, q=x["q"][:, heads], **{n: x[n][:, kv] for n in ("k", "v", "kp", "vp")})
    check((o[:, heads], lse[heads]), reference(part, 128 ** -0.5, True))


@gpu
def test_rope_cache_and_both_decodes_together():
    """A serving path: turn a prompt's and three continuations' keys by their (time, height, width)
    positions, append them to the cache (the prompt's pages shared by all), decode over the cache;
    then read the cache back and decode with the prompt as a shared prefix.  The two decodes see
    the same values, so they agree to their roundings."""
    H, Hkv, d, page, prompt = 8, 2, 128, 64, 256  # the prompt ends with its page
    own = [3, 70, 1]
    table = fa.rope_table(d, (16, 24, 24))
    g = torch.Generator().manual_seed(12)
    total = prompt + sum(own)
    qs, ks, vs = (torch.randn(total, h, d, generator=g).bfloat16().cuda() for h in (H, Hkv, Hkv))
    pos = torch.cat([torch.arange(prompt)] + [prompt + torch.arange(n) for n in own])
    pos = torch.stack([pos, pos // 16, pos % 16]).to(torch.int32).cuda()
    q, k = fa.rope(qs, ks, pos, table)
    # pages: 4 of the prompt, then each continuation's
    cache = fa.new_cache(16, page, Hkv, d)
    pages = torch.full((4, 8), -1, dtype=torch.int32)
    pages[:, :4] = torch.tensor([9, 3, 12, 0])
    for b, mine in enumerate(([5], [1, 7], [2])):
        pages[1 + b, 4:4 + len(mine)] = torch.tensor(mine)
    lens = torch.tensor([prompt] + [prompt + n for n in own], dtype=torch.int32)
    fa.cache_append(cache, k, vs, cu([prompt] + own).cuda(), lens.cuda(), pages.cuda(), prompt)
    # the last token of each continuation asks
    ends = [prompt + sum(own[:b + 1]) - 1 for b in range(3)]
    qd = q[ends].contiguous()
    ones, tab, n = cu([1] * 3).cuda(), pages[1:].contiguous().cuda(), lens[1:].contiguous().cuda()
    a = fa.forward_decode_cache(qd, cache, ones, n, tab, 1, prompt + max(own), causal=True)
    kr, vr = fa.cache_read(cache, cu(lens[1:].tolist()).cuda(), tab, prompt + max(own),
                           int(lens[1:].sum()))
    at = np.cumsum([0] + lens[1:].tolist())
    kp, vp = (t[:prompt].contiguous() for t in (kr, vr))
    ko, vo = (torch.cat([t[at[b] + prompt:at[b + 1]] for b in range(3)]) for t in (kr, vr))
    b = fa.forward_decode_shared(qd, kp, vp, ko, vo, ones, cu(own).cuda(), cu([3]).cuda(),
                                 cu([prompt]).cuda(), 1, max(own), 3, prompt, causal=True)
    fa.fa_device_status()
    x = dict(q=qd.cpu(), k=ko.cpu(), v=vo.cpu(), kp=kp.cpu(), vp=vp.cpu(), cu_q=cu([1] * 3),
             cu_k=cu(own), cu_g=cu([3]), cu_p=cu([prompt]))
    ref = reference(x, d ** -0.5, True)
    for got in (a, b):
        check(got, ref)


# ------------------------------------------------------------------------------ refusals (CPU)

@pytest.fixture(scope="module")
def lib():
    from exact_attention_25_gb300 import _lib, build

    build.build()
    return _lib.load(_lib.LIB_PATH)


@pytest.mark.parametrize("kw, code", [
    (dict(d=96), -2), (dict(B=0), -1), (dict(Hkv=0), -1), (dict(H=3), -1), (dict(groups=0), -1),
    (dict(tq=0), -1), (dict(tk=0), -1), (dict(tp=0), -1), (dict(mq=0), -1), (dict(mk=0), -1),
    (dict(mg=0), -1), (dict(mp=0), -1), (dict(H=129, Hkv=1), -1), (dict(causal=2), -1),
    (dict(scale=float("nan")), -1), (dict(ctas=0), -1), (dict(ctas=1025), -1), (dict(q=0), -1),
    (dict(kp=0), -1), (dict(vp=0), -1), (dict(k=0), -1), (dict(o=0), -1), (dict(cq=0), -1),
    (dict(ck=0), -1), (dict(cg=0), -1), (dict(cp=0), -1), (dict(q=0x10008), -3),
    (dict(vp=0x30008), -3), (dict(lse=0x70002), -3), (dict(cg=0x92002), -3), (dict(ws=0), -4),
    (dict(wsb=100), -4), (dict(ws=0xA0004), -3), (dict(tp=1 << 26, H=4, Hkv=4, d=64), -7),
    (dict(tq=1 << 25), -7), (dict(B=1 << 22, tq=1 << 10, mq=1 << 10, H=4), -7),
])
def test_decode_shared_refuses(lib, kw, code):
    a = dict(q=0x10000, kp=0x20000, vp=0x30000, k=0x40000, v=0x50000, o=0x60000, lse=0x70000,
             cq=0x90000, ck=0x91000, cg=0x92000, cp=0x93000, B=2, groups=1, mq=1, mk=10, mg=2, mp=100,
             tq=2, tk=20, tp=100, H=4, Hkv=2, d=64, scale=0.1, causal=0, ctas=2, ws=0xA0000,
             wsb=1 << 30)
    a.update(kw)
    vp = ctypes.c_void_p
    rc = lib.fa_fwd_decode_shared(
        *(vp(a[n]) for n in ("q", "kp", "vp", "k", "v", "o", "lse", "cq", "ck", "cg", "cp")),
        *(a[n] for n in ("B", "groups", "mq", "mk", "mg", "mp", "tq", "tk", "tp", "H", "Hkv", "d")),
        ctypes.c_float(a["scale"]), a["causal"], a["ctas"], vp(a["ws"]), a["wsb"], None)
    assert rc == code


def test_workspace_of_the_shared_decode(lib):
    w = lib.fa_decode_shared_workspace_bytes
    assert w(0, 4, 64, 1) == 0 and w(4, 4, 96, 1) == 0 and w(4, 4, 64, 0) == 0 and w(4, 4, 64, 1025) == 0
    for T, H, d, c in ((1, 1, 64, 1), (7, 32, 128, 152)):
        rows = 2 * T * H + 256 * c
        assert rows * (d + 1) * 4 <= w(T, H, d, c) <= rows * (d + 1) * 4 + 512
