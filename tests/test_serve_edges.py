"""Serving operators at their edges: waits that run out, the bounds-checked library, causal masks
of sequences longer than their row of the page table, many key/value heads, calls that several streams
make at once, captured work of two streams, tensors that overlap, and what the binding refuses."""
import ctypes
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import exact_attention_25_gb300 as fa
from exact_attention_25_gb300 import _lib
from tests import test_cache, test_decode_cache, test_decode_shared
from tests.serve_util import attention_rows
from tests.test_cache import cu, table_for

gpu = pytest.mark.gpu
i32 = lambda *v: torch.tensor(v, dtype=torch.int32)  # noqa: E731


# ------------------------------------------------------------------------------ waits that run out

@pytest.fixture
def short_waits():
    lib = fa.load()
    fa.fa_set_wait_limit_ns(20_000_000)  # 20 ms
    yield lib
    lib.fa_debug_set_flags(0)
    fa.fa_set_wait_limit_ns(2_000_000_000)


def expires(lib, call):
    """With the first block's copy announced and never made (a test hook) the waits expire, the call
    ends and reports; afterwards the same call works."""
    want = call()
    fa.fa_device_status()
    lib.fa_debug_set_flags(1)
    call()
    with pytest.raises(fa.FaError) as e:
        fa.fa_device_status()
    assert e.value.code == -6 and "site" in _lib.last_error()
    lib.fa_debug_set_flags(0)
    got = call()
    fa.fa_device_status()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def cache_call(lens_q, lens_k, H, Hkv, d, page, causal, ctas, seed):
    table, pool = table_for(lens_k, page, 1, seed)
    cache = test_decode_cache.to_cache(*test_decode_cache.random_cache(pool, Hkv, page, d, seed))
    q = torch.randn(sum(lens_q), H, d, generator=torch.Generator().manual_seed(seed)).bfloat16().cuda()
    a = (cu(lens_q).cuda(), i32(*lens_k).cuda(), table.cuda(), max(lens_q), max(lens_k), d ** -0.5,
         causal, ctas)
    return lambda: fa.forward_decode_cache(q, cache, *a)


@gpu
@pytest.mark.parametrize("d", [64, 128])
def test_cache_decode_wait_expires_and_context_survives(short_waits, d):
    expires(short_waits, cache_call([1, 2], [300, 700], 8, 2, d, 64, True, 5, 1))


@gpu
@pytest.mark.parametrize("d", [64, 128])
def test_shared_decode_wait_expires_and_context_survives(short_waits, d):
    x = test_decode_shared.make([1, 2, 1], [30, 200, 5], [0, 3], [900], 8, 2, d, 2)
    expires(short_waits, lambda: test_decode_shared.run(x, 0.1, True, 6))


# ------------------------------------------------------------------------------ checked library

@pytest.fixture(scope="module")
def checked():
    if not os.path.exists(_lib.LIB_CHECKED_PATH):
        from exact_attention_25_gb300 import build

        build.build(checked=True)
    return _lib.LIB_CHECKED_PATH


def checked_calls(d, dtype):
    """One call of every serving operator, as functions of nothing that return tensors."""
    g = torch.Generator().manual_seed(d)
    rnd = lambda *s: torch.randn(*s, generator=g).to(dtype).cuda()  # noqa: E731
    pos = torch.randint(-50, 50, (2, 37), generator=g, dtype=torch.int32).cuda()
    q, k = rnd(37, 6, d), rnd(37, 2, d)
    table = fa.rope_table(d, (8, 16))
    lens, page = [20, 17], 16
    tab, pool = table_for(lens, page, 1, 3)
    kn, vn = rnd(37, 2, d), rnd(37, 2, d)

    def append():
        c = fa.new_cache(pool, page, 2, d)
        fa.cache_append(c, kn, vn, cu(lens).cuda(), i32(*lens).cuda(), tab.cuda(), 20)
        return [t.view(torch.uint8) for t in c]

    def read():
        c = test_decode_cache.to_cache(*test_decode_cache.random_cache(pool, 2, page, d, 5))
        return fa.cache_read(c, cu(lens).cuda(), tab.cuda(), 20, 37, dtype)

    x = test_decode_shared.make([1, 2, 1], [30, 200, 5], [0, 3], [300], 8, 2, d, 2)
    return {"rope": lambda: fa.rope(q, k, pos, table), "append": append, "read": read,
            "decode_cache": cache_call([1, 2], [300, 700], 8, 2, d, 64, True, 5, 1),
            "decode_shared": lambda: test_decode_shared.run(x, 0.1, True, 6)}


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d", [64, 128])
def test_checked_library_gives_the_same_bits(checked, d, dtype):
    calls = checked_calls(d, dtype)
    want = {}
    with _lib.library(_lib.LIB_PATH):
        for n, f in calls.items():
            want[n] = [t.clone() for t in f()]
        fa.fa_device_status()
    with _lib.library(checked):
        assert fa.fa_checked_build()
        for n, f in calls.items():
            got = f()
            fa.fa_device_status()
            for a, b in zip(got, want[n]):
                assert torch.equal(a, b), n


@gpu
@pytest.mark.parametrize("name", ["rope", "append", "read", "decode_cache", "decode_shared"])
@pytest.mark.parametrize("d", [64, 128])
def test_checked_library_catches_shrunk_extents(checked, d, name):
    with _lib.library(checked) as lib:
        call = checked_calls(d, torch.bfloat16)[name]
        lib.fa_debug_set_flags(2)  # every extent one row short
        try:
            call()
            with pytest.raises(fa.FaError) as e:
                fa.fa_device_status()
            assert e.value.code == -9
        finally:
            lib.fa_debug_set_flags(0)
        call()
        fa.fa_device_status()


# ------------------------------------------------------------------------------ tables that end early

@gpu
@pytest.mark.parametrize("ctas", [1, 3])
@pytest.mark.parametrize("d", [64, 128])
def test_keys_past_the_table_are_left_out_and_counted_by_the_mask(d, ctas):
    """Sequences longer than max_pages * page_size: the mask of query i still ends at key
    length - queries + i, of which the table holds the first ones."""
    H, Hkv, page, room = 4, 2, 16, 160
    lens_q, lens_k = [6, 3, 9], [162, 400, 163]
    table, pool = table_for([room] * 3, page, 1, 8)
    codes, exps = test_decode_cache.random_cache(pool, Hkv, page, d, 8)
    q = torch.randn(sum(lens_q), H, d, generator=torch.Generator().manual_seed(8)).bfloat16()
    got = fa.forward_decode_cache(q.cuda(), test_decode_cache.to_cache(codes, exps), cu(lens_q).cuda(),
                                  i32(*lens_k).cuda(), table.cuda(), max(lens_q), 1000, 0.1, True, ctas)
    fa.fa_device_status()
    T = sum(lens_q)
    ref = [np.zeros((T, H, d)), np.zeros((H, T)), np.zeros((T, H, d)), np.zeros((H, T)), np.zeros((T, H, d))]
    t = 0
    for b, (n, nk) in enumerate(zip(lens_q, lens_k)):
        for h in range(H):
            k, v = (test_decode_cache.sequence(codes, exps, z, table, b, h // 2, room, page) for z in (0, 1))
            o, lse, pv, mag, low = attention_rows(
                q[t:t + n, h].double().numpy(), k, v, 0.1, True, nk - n,
                test_decode_cache.row_scale(exps[1], table, b, h // 2, room, page))
            ref[0][t:t + n, h], ref[1][h, t:t + n] = o, lse
            ref[2][t:t + n, h], ref[3][h, t:t + n], ref[4][t:t + n, h] = pv, mag, low
        t += n
    test_decode_cache._check(got, ref)


# ------------------------------------------------------------------------------ head layouts

@gpu
@pytest.mark.parametrize("H, Hkv, d", [(96, 96, 64), (80, 80, 128), (5, 5, 64), (160, 160, 64), (21, 7, 128)])
def test_shared_decode_of_many_heads(H, Hkv, d):
    """More heads than go round in the thread blocks: several to a line."""
    x = test_decode_shared.make([1, 1, 2], [20, 0, 150], [0, 2, 3], [300, 129], H, Hkv, d, H)
    got = test_decode_shared.run(x, 0.1, True)
    fa.fa_device_status()
    test_decode_shared.check(got, test_decode_shared.reference(x, 0.1, True))


# ------------------------------------------------------------------------------ odd values of seen keys

@gpu
@pytest.mark.parametrize("ctas", [None, 1, 7])
@pytest.mark.parametrize("nq", [1, 9, 40])
@pytest.mark.parametrize("d", [64, 128])
def test_infinities_of_seen_keys_come_out(d, nq, ctas):
    """V of keys that every query sees holds infinities and a NaN, in the prefix and in own keys: they
    reach their columns and no other, whatever the number of rows of a tile."""
    x = test_decode_shared.make([nq, nq], [300, 70], [0, 2], [500], 4, 2, d, nq)
    at = {("vp", 3): (float("inf"), 5), ("vp", 450): (float("-inf"), 6), ("vp", 260): (float("nan"), 7),
          ("v", 40): (float("inf"), 8), ("v", 200): (float("-inf"), 9), ("v", 310): (float("inf"), 10)}
    clean = {n: t.clone() if torch.is_tensor(t) else t for n, t in x.items()}
    for (name, j), (val, c) in at.items():
        x[name][j, 1, c] = val
        clean[name][j, 1, c] = 0.0
    o, lse = test_decode_shared.run(x, 0.1, False, ctas)
    fa.fa_device_status()
    ref = test_decode_shared.reference(clean, 0.1, False)
    for (name, j), (val, c) in at.items():
        rows = slice(0, 2 * nq) if name == "vp" else slice(0, nq) if j < 300 else slice(nq, 2 * nq)
        got = o[rows, 2:, c].float().cpu()  # heads 2, 3 read key/value head 1
        assert (torch.isnan(got) if val != val else got == val).all(), (name, j)
        ref[0][rows, 2:, c] = val
    keep = ~(np.isinf(ref[0]) | np.isnan(ref[0]))
    got = torch.where(torch.tensor(keep), o.double().cpu(), torch.tensor(0.0, dtype=torch.float64))
    ref[0][~keep] = 0.0
    test_decode_shared.check((got, lse), ref)


@gpu
@pytest.mark.parametrize("ctas", [None, 3, 152])
@pytest.mark.parametrize("d", [64, 128])
def test_units_of_few_and_many_rows_side_by_side(d, ctas):
    """Groups whose tiles hold 32 rows, a little more, and several tiles; own keys of one to 33 tokens."""
    lens_q = [1, 2, 8, 1, 4, 4, 33, 1, 9, 30]
    lens_k = [200, 1, 130, 0, 127, 129, 40, 1000, 9, 31]
    x = test_decode_shared.make(lens_q, lens_k, [0, 3, 6, 8, 10], [700, 129, 0, 1500], 8, 2, d, 21)
    for causal in (False, True):
        got = test_decode_shared.run(x, 0.1, causal, ctas)
        fa.fa_device_status()
        test_decode_shared.check(got, test_decode_shared.reference(x, 0.1, causal))


@gpu
def test_shared_decode_of_one_long_and_many_short_sequences():
    """Nine single tokens in a group and a sequence of 1100 tokens outside it."""
    x = test_decode_shared.make([1] * 9 + [1100], [60, 1, 0, 300, 5, 7, 128, 64, 2, 1100], [0, 9], [200], 32, 1, 64, 5)
    got = test_decode_shared.run(x, 0.1, True)
    fa.fa_device_status()
    few = 9
    part = {n: x[n] for n in ("k", "v", "kp", "vp", "cu_g", "cu_p")}
    part.update(q=x["q"][:few], cu_q=x["cu_q"][:few + 1], cu_k=x["cu_k"][:few + 1])
    ref = test_decode_shared.reference(part, 0.1, True)
    test_decode_shared.check((got[0][:few], got[1][:, :few]), ref)
    last = x["q"][few:few + 1100]
    heads = slice(0, 2)
    tail = dict(q=last[:, heads], k=x["k"][-1100:], v=x["v"][-1100:], kp=x["kp"], vp=x["vp"],
                cu_q=cu([1100]), cu_k=cu([1100]), cu_g=i32(1, 1), cu_p=i32(0, 200))
    ref = test_decode_shared.reference(tail, 0.1, True)
    test_decode_shared.check((got[0][few:, heads], got[1][heads, few:]), ref)


# ------------------------------------------------------------------------------ large appends

@gpu
@pytest.mark.parametrize("strided", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_a_large_append_equals_small_ones(dtype, d, strided):
    """A batch whose grid takes k and v in turn, against its sequences one by one, whose grids take
    them side by side; a row of every kind of value in both."""
    B, Hkv, page = 40, 6, 64
    lens = [70 + 3 * b for b in range(B)]
    table, pool = table_for(lens, page, 1, 5)
    g = torch.Generator().manual_seed(d)
    T = sum(lens)
    x = torch.randn(2, T, Hkv, d + (8 if strided else 0), generator=g).to(dtype).cuda()[..., :d]
    x[0, 5] = 0.0
    x[1, T - 1, 2, 3] = float("inf")
    x[0, T // 2, 1, 7] = float("nan")
    starts = np.cumsum([0] + lens)
    many, few = fa.new_cache(pool, page, Hkv, d), fa.new_cache(pool, page, Hkv, d)
    fa.cache_append(many, x[0], x[1], cu(lens).cuda(), i32(*lens).cuda(), table.cuda(), max(lens))
    for b, n in enumerate(lens):
        k, v = (t[starts[b]:starts[b + 1]] for t in x)
        fa.cache_append(few, k, v, i32(0, n).cuda(), i32(n).cuda(), table[b:b + 1].cuda(), n)
    fa.fa_device_status()
    for a, b in zip(many, few):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


# ------------------------------------------------------------------------------ streams and graphs

@gpu
def test_calls_on_several_streams_at_once():
    """The same calls, made by four streams at once, give what they give alone."""
    x = test_decode_shared.make([1, 1, 2], [40, 7, 300], [0, 3], [700], 8, 2, 128, 4)
    dev = {n: t.cuda() for n, t in x.items() if n != "sizes"}
    shared = lambda s=None: fa.forward_decode_shared(  # noqa: E731
        dev["q"], dev["kp"], dev["vp"], dev["k"], dev["v"], dev["cu_q"], dev["cu_k"], dev["cu_g"],
        dev["cu_p"], *x["sizes"], 0.1, True, None, s)
    cache = cache_call([1, 2], [3000, 700], 8, 2, 128, 64, True, None, 1)
    pos = torch.arange(37, dtype=torch.int32)[None].cuda()
    q = torch.randn(37, 6, 128).bfloat16().cuda()
    table = fa.rope_table(128, (64,))
    want = shared() + cache() + (fa.rope(q, None, pos, table)[0],)
    streams = [torch.cuda.Stream() for _ in range(4)]
    torch.cuda.synchronize()
    got = []
    for _ in range(10):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(shared() + cache() + (fa.rope(q, None, pos, table)[0],))
    torch.cuda.synchronize()
    fa.fa_device_status()
    for g in got:
        for a, b in zip(g, want):
            assert torch.equal(a, b)


@gpu
def test_capture_of_work_that_forks_and_joins():
    """Inputs made on another stream inside the capture: a call's first kernel then follows an event,
    not a kernel of its own stream."""
    d, page = 128, 64
    tab, pool = table_for([200, 90], page, 1, 1)
    tab = tab.cuda()
    cache = fa.new_cache(pool, page, 2, d)
    src = torch.randn(290, 2, d).bfloat16().cuda()
    k, pos = torch.empty_like(src), torch.arange(290, dtype=torch.int32)[None].cuda()
    qs, q = torch.randn(2, 8, d).bfloat16().cuda(), torch.empty(2, 8, d, dtype=torch.bfloat16).cuda()
    starts, ones, n = cu([200, 90]).cuda(), cu([1, 1]).cuda(), i32(0, 0).cuda()
    lens = i32(200, 90).cuda()
    table = fa.rope_table(d, (64,))
    side = torch.cuda.Stream()

    def step():
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            k.copy_(src)
            fa.fa_rope(k, None, k, None, pos, table)
        n.copy_(lens)
        q.copy_(qs)
        main.wait_stream(side)
        fa.cache_append(cache, k, src, starts, n, tab, 200)
        o, lse = fa.forward_decode_cache(q, cache, ones, n, tab, 1, 200, causal=True)
        side.wait_stream(main)
        with torch.cuda.stream(side):
            back = fa.cache_read(cache, starts, tab, 200, 290)
        main.wait_stream(side)
        return o, lse, *back

    want = [t.clone() for t in step()]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for seed in range(3):
        for t in out + (k, q):
            t.fill_(7.0)
        n.zero_()
        for t in cache:
            t.view(torch.uint8).fill_(127)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert torch.equal(a, b)
    fa.fa_device_status()


FIRST_CALLS = """
import torch, exact_attention_25_gb300 as fa
i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")
q, k = torch.randn(2, 4, 64, device="cuda").bfloat16(), torch.randn(300, 2, 64, device="cuda").bfloat16()
v, pos, table = torch.randn_like(k), i32(0, 1)[None], fa.rope_table(64, (32,))
cache, pages = fa.new_cache(10, 64, 2, 64), torch.arange(10, dtype=torch.int32, device="cuda").view(2, 5)
cu, n, ones, two, p = i32(0, 150, 300), i32(150, 150), i32(0, 1, 2), i32(0, 2), i32(0, 300)
torch.cuda.synchronize()
for f in (lambda: fa.rope(q, k[:2].contiguous(), pos, table),
          lambda: fa.cache_append(cache, k, v, cu, n, pages, 150),
          lambda: fa.cache_read(cache, cu, pages, 150, 300),
          lambda: fa.forward_decode_cache(q, cache, ones, n, pages, 1, 150),
          lambda: fa.forward_decode_shared(q, k, v, k, v, ones, cu, two, p, 1, 150, 2, 300)):
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        r = f()
    g.replay()
    torch.cuda.synchronize()
    for a, b in zip(r or (), f() or ()):
        assert torch.equal(a, b)
fa.fa_device_status()
"""


@gpu
def test_first_calls_of_a_process_may_be_captured():
    """Nothing has run before: the first call of every operator is made inside a capture."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS], cwd=root, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-2000:]


# ------------------------------------------------------------------------------ far offsets

@gpu
def test_pages_more_than_32_bits_into_the_cache():
    """Sequences whose pages lie at the two ends of a pool of more than 2^32 codes."""
    Hkv, d, page, H = 8, 128, 64, 16
    pool = 2 ** 32 // (Hkv * page * d) + 8
    big = fa.new_cache(pool, page, Hkv, d)
    assert big.k.numel() > 2 ** 32
    lens = [150, 200]
    near = torch.tensor([[0, 1, 2, -1], [3, 4, 5, 6]], dtype=torch.int32)
    far = torch.tensor([[pool - 1, 0, pool - 2, -1], [pool - 7, pool - 4, 1, pool - 3]], dtype=torch.int32)
    small = fa.new_cache(7, page, Hkv, d)
    g = torch.Generator().manual_seed(1)
    k, v = (torch.randn(350, Hkv, d, generator=g).bfloat16().cuda() for _ in range(2))
    q = torch.randn(3, H, d, generator=g).bfloat16().cuda()
    n, got = i32(*lens).cuda(), []
    for cache, table in ((small, near.cuda()), (big, far.cuda())):
        fa.cache_append(cache, k, v, cu(lens).cuda(), n, table, 200)
        back = fa.cache_read(cache, cu(lens).cuda(), table, 200, 350)
        out = fa.forward_decode_cache(q, cache, i32(0, 1, 3).cuda(), n, table, 2, 200, causal=True)
        got.append((*back, *out))
    fa.fa_device_status()
    for a, b in zip(*got):
        assert torch.equal(a, b)


@gpu
def test_rope_of_more_than_32_bits_of_elements():
    """q of more than 2^32 elements, in place: tokens at both ends turn as they do alone."""
    H, d = 64, 128
    total = 2 ** 32 // (H * d) + 5
    q = torch.empty(total, H, d, dtype=torch.bfloat16, device="cuda")
    ends = torch.tensor([0, 1, total // 2, total - 2, total - 1], device="cuda")
    part = torch.randn(5, H, d, generator=torch.Generator().manual_seed(2)).bfloat16().cuda()
    q.zero_()
    q[ends] = part
    pos = torch.arange(total, dtype=torch.int32, device="cuda")[None] * 3
    table = fa.rope_table(d, (64,))
    fa.fa_rope(q, None, q, None, pos, table)
    want, _ = fa.rope(part, None, pos[:, ends].contiguous(), table)
    fa.fa_device_status()
    assert torch.equal(q[ends], want)


# ------------------------------------------------------------------------------ overlap (CPU)

@pytest.fixture(scope="module")
def lib():
    from exact_attention_25_gb300 import build

    build.build()
    return _lib.load(_lib.LIB_PATH)


@pytest.mark.parametrize("kw", [dict(kc=0x40000 - 64), dict(ke=0x30000), dict(k=0x30000), dict(v=0x60000),
                                dict(ve=0x50010)])
def test_append_refuses_overlap(lib, kw):
    assert test_cache.append(lib, {**test_cache.BASE, **kw}) == -1
    assert b"overlap" in lib.fa_last_error()


@pytest.mark.parametrize("kw", [dict(k=0x30000), dict(v=0x10000), dict(v=0x50000), dict(k=0x20000 - 16)])
def test_read_refuses_overlap(lib, kw):
    assert test_cache.read(lib, {**test_cache.BASE, **kw}) == -1
    assert b"overlap" in lib.fa_last_error()


@pytest.mark.parametrize("kw", [dict(o=0x10000), dict(o=0x30000), dict(o=0x60000), dict(lse=0x70000), dict(o=0x91000),
                                dict(ws=0x10000), dict(ws=0x70000), dict(lse=0x92000), dict(ws=0x93000)])
def test_cache_decode_refuses_overlap(lib, kw):
    a = dict(q=0x10000, kc=0x30000, vc=0x40000, ke=0x50000, ve=0x60000, o=0x70000, lse=0x80000,
             cu=0x91000, n=0x92000, table=0x93000, ws=0xA0000)
    a.update(kw)
    vp = ctypes.c_void_p
    rc = lib.fa_fwd_decode_cache(
        *(vp(a[n]) for n in ("q", "kc", "vc", "ke", "ve", "o", "lse", "cu", "n", "table")), 1, 1, 100, 1,
        8, 8, 16, 4, 2, 64, ctypes.c_float(0.1), 0, 2, vp(a["ws"]), 1 << 20, None)
    assert rc == -1 and b"overlap" in lib.fa_last_error()


@pytest.mark.parametrize("kw", [dict(o=0x10000), dict(o=0x20000), dict(o=0x50000), dict(lse=0x60000),
                                dict(ws=0x40000), dict(ws=0x60000), dict(lse=0x92000), dict(o=0x93000)])
def test_shared_decode_refuses_overlap(lib, kw):
    a = dict(q=0x10000, kp=0x20000, vp=0x30000, k=0x40000, v=0x50000, o=0x60000, lse=0x70000,
             cq=0x90000, ck=0x91000, cg=0x92000, cp=0x93000, ws=0xA0000)
    a.update(kw)
    vp = ctypes.c_void_p
    rc = lib.fa_fwd_decode_shared(
        *(vp(a[n]) for n in ("q", "kp", "vp", "k", "v", "o", "lse", "cq", "ck", "cg", "cp")),
        2, 1, 1, 10, 2, 100, 2, 20, 100, 4, 2, 64, ctypes.c_float(0.1), 0, 2, vp(a["ws"]), 1 << 30, None)
    assert rc == -1 and b"overlap" in lib.fa_last_error()


# ------------------------------------------------------------------------------ the binding (CPU)

def test_rope_table_takes_any_sequence_of_sections():
    assert fa.rope_table(64, [8, 24]) is fa.rope_table(64, (8, 24))
    t = fa.rope_table(128, np.array([16, 24, 24]))
    assert t.pairs == 64 and t.axes == 3 and t.axis == (0,) * 16 + (1,) * 24 + (2,) * 24


def test_binding_refuses_types_and_shapes():
    q, kv = torch.zeros(2, 4, 64).bfloat16(), torch.zeros(9, 2, 64).bfloat16()
    cache = fa.new_cache(2, 16, 2, 64, device="cpu")
    tab, ones, n = torch.zeros(2, 1, dtype=torch.int32), i32(0, 1, 2), i32(3, 4)
    dec = lambda **k: fa.forward_decode_cache(**{**dict(  # noqa: E731
        q=q, cache=cache, cu_seqlens_q=ones, seqlens_k=n, page_table=tab, max_seqlen_q=1, max_seqlen_k=9), **k})
    for kw, err in ((dict(q=q.float()), TypeError), (dict(q=q[0]), ValueError), (dict(q=q.transpose(0, 1)), ValueError),
                    (dict(cu_seqlens_q=ones[:2]), ValueError), (dict(cu_seqlens_q=ones.long()), TypeError),
                    (dict(seqlens_k=i32(1)), ValueError), (dict(page_table=tab[0]), ValueError),
                    (dict(page_table=tab.long()), TypeError), (dict(max_seqlen_q=2 ** 40), ValueError),
                    (dict(max_seqlen_k="9"), TypeError), (dict(scale="x"), TypeError), (dict(q=None), AttributeError),
                    (dict(cache=cache._replace(k=cache.k[:, :, :, :32])), ValueError), (dict(), ValueError)):
        with pytest.raises(err):
            dec(**kw)
    sh = lambda **k: fa.forward_decode_shared(**{**dict(  # noqa: E731
        q=q, k_prefix=kv, v_prefix=kv, k=kv, v=kv, cu_seqlens_q=ones, cu_seqlens_k=i32(0, 4, 9),
        cu_groups=i32(0, 2), cu_seqlens_p=i32(0, 9), max_seqlen_q=1, max_seqlen_k=5, max_group_q=2,
        max_seqlen_p=9), **k})
    for kw, err in ((dict(k=kv.float(), v=kv.float()), ValueError), (dict(v=kv[:, :1]), ValueError),
                    (dict(k_prefix=kv[:, :, :32]), ValueError), (dict(cu_seqlens_k=i32(0, 9)), ValueError),
                    (dict(cu_groups=i32(0, 2)[None]), ValueError), (dict(cu_seqlens_p=i32(0, 4, 9)), ValueError),
                    (dict(), ValueError)):
        with pytest.raises(err):
            sh(**kw)
    with pytest.raises(TypeError):
        fa.cache_read(cache, i32(0, 3, 7), tab, 4, 7, dtype=torch.float16)
    with pytest.raises(ValueError):
        fa.fa_fwd_decode_cache(q, cache, None, None, ones, n, tab, 1, 9, 0.1, False, 1, None)
    with pytest.raises(ValueError):
        fa.fa_fwd_decode_cache(q, cache, q, None, ones, n, tab, 1, 9, 0.1, False, 0, None)


@gpu
def test_binding_refuses_mixed_devices_and_foreign_outputs():
    q, k = torch.zeros(4, 2, 64).bfloat16().cuda(), torch.zeros(4, 1, 64).bfloat16().cuda()
    pos, table = torch.zeros(1, 4, dtype=torch.int32), fa.rope_table(64, (32,))
    with pytest.raises(ValueError):
        fa.rope(q, k, pos, table)
    with pytest.raises(ValueError):
        fa.rope(q, k.cpu(), pos.cuda(), table)
    with pytest.raises(ValueError):
        fa.rope(q, k.float(), pos.cuda(), table)
    with pytest.raises(ValueError):
        fa.fa_rope(q, k, q, q, pos.cuda(), table)
    with pytest.raises(ValueError):
        fa.rope(q[:, :, :32].contiguous(), k, pos.cuda(), table)
    with pytest.raises(ValueError):
        fa.rope(q, k, pos.cuda(), fa.rope_table(64, (16, 16)))  # two axes, one row of positions
    with pytest.raises(fa.FaError):
        fa.fa_rope(k, k.clone(), k, k, pos.cuda(), table)  # both outputs one tensor
    cache = fa.new_cache(2, 16, 2, 64)
    tab, ones, n = torch.zeros(4, 1, dtype=torch.int32).cuda(), cu([1] * 4).cuda(), i32(1, 2, 3, 4).cuda()
    with pytest.raises(ValueError):
        fa.forward_decode_cache(q, fa.new_cache(2, 16, 2, 64, device="cpu"), ones, n, tab, 1, 4)
    with pytest.raises(ValueError):
        fa.forward_decode_cache(q, cache, ones.cpu(), n, tab, 1, 4)
    with pytest.raises(fa.FaError):  # in place
        fa.fa_fwd_decode_cache(q, cache, q, None, ones, n, tab, 1, 4, 0.1, False, 1, None)
