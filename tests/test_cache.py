"""The paged e4m3 cache: fa_cache_append against the definition of its codes and exponents bit for
bit, fa_cache_read exactly, over types, page sizes, strides, empty and single-token sequences;
infinities, NaNs, zeros and extreme sizes; bad table entries; rows and pages that must stay as
they are; refusals."""
import ctypes

import numpy as np
import pytest
import torch

import exact_attention_25_gb300 as fa
from tests.gpu_util import guarded_empty
from tests.serve_util import quantise_row, values

gpu = pytest.mark.gpu


def cu(lens):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32)


def table_for(lens, page, spare, seed):
    """A page table with every sequence's pages in random order, and the pool's size."""
    need = [-(-n // page) for n in lens]
    order = np.random.RandomState(seed).permutation(sum(need) + spare)
    t = np.full((len(lens), max(max(need), 1)), 10 ** 9, np.int32)  # unused entries: no page
    at = 0
    for b, n in enumerate(need):
        t[b, :n] = order[at:at + n]
        at += n
    return torch.tensor(t), sum(need) + spare


CASES = {
    # name: (new tokens, cached before, Hkv, d, page, dtype)
    "one_token": ([1], [0], 1, 128, 16, torch.bfloat16),
    "one_token_each": ([1, 1, 1, 1], [63, 64, 0, 200], 8, 128, 64, torch.bfloat16),
    "ragged": ([17, 0, 33, 1, 130], [5, 9, 0, 15, 31], 3, 128, 16, torch.bfloat16),
    "fp32_d64": ([40, 2, 0], [1, 0, 3], 2, 64, 32, torch.float32),
    "fp32": ([9, 70], [120, 0], 5, 128, 128, torch.float32),
    "bf16_d64": ([100, 1], [30, 1023], 1, 64, 1024, torch.bfloat16),
}


@gpu
@pytest.mark.parametrize("case", list(CASES))
def test_append_then_read(case):
    new, old, Hkv, d, page, dtype = CASES[case]
    lens = [a + b for a, b in zip(new, old)]
    T = sum(new)
    table, pool = table_for(lens, page, 2, 3)
    g = torch.Generator().manual_seed(len(case))
    size = torch.exp(3 * torch.randn(T, Hkv, 1, generator=g))
    k, v = ((torch.randn(T, Hkv, d, generator=g) * size).to(dtype) for _ in range(2))
    if T > 1:
        k[0, 0] = 0.0                       # a row of zeros
        v[1, 0, 3], v[1, 0, 7] = float("inf"), float("nan")
        k[1, -1] *= 2.0 ** 100              # far from 1, and (below) under the smallest scale
        v[0, -1] = (v[0, -1].double() * 2.0 ** -125).to(dtype)
        k[T - 1, 0] = 448.0 * torch.where(torch.arange(d) % 2 == 0, 1.0, -0.5)
    cache = fa.new_cache(pool, page, Hkv, d)
    fill = 0x5A
    for t in cache:
        t.view(torch.uint8).fill_(fill)
    seqlens = torch.tensor(lens, dtype=torch.int32)
    fa.cache_append(cache, k.cuda(), v.cuda(), cu(new).cuda(), seqlens.cuda(), table.cuda(),
                    max(new))
    fa.fa_device_status()
    host = [t.view(torch.uint8).cpu().numpy() for t in cache]
    want = [np.full_like(h, fill) for h in host]
    at = 0
    for b, n in enumerate(new):
        for i in range(n):
            pos = old[b] + i
            p, r = int(table[b, pos // page]), pos % page
            for hk in range(Hkv):
                for z, x in ((0, k), (1, v)):
                    c, e = quantise_row(x[at + i, hk].double().numpy())
                    want[z][p, hk, r], want[2 + z][p, hk, r] = c, e
        at += n
    for z in range(2):
        same = (host[z] & 127 == 127) & (want[z] & 127 == 127)  # any NaN code is NaN
        assert (same | (host[z] == want[z])).all()
        assert (host[2 + z] == want[2 + z]).all()
    # read back all of it (the rows before the new ones hold the fill's values)
    for out in (torch.bfloat16, torch.float32):
        kr, vr = fa.cache_read(cache, cu(lens).cuda(), table.cuda(), max(lens), sum(lens), out)
        row = 0
        for b, n in enumerate(lens):
            for i in range(n):
                p, r = int(table[b, i // page]), i % page
                for got, z in ((kr, 0), (vr, 1)):
                    x = torch.tensor(values(want[z][p, :, r], want[2 + z][p, :, r]))
                    assert torch.equal(torch.nan_to_num(x.to(out), nan=77.0),
                                       torch.nan_to_num(got[row].cpu(), nan=77.0))
                row += 1


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_quantisation_at_every_kind_of_value(dtype):
    """Rows whose largest value sits on either side of a power-of-two scale, values midway
    between codes (ties), and every exponent of the type."""
    d = 64
    rows = []
    for top in (448.0, 448.0 * (1 + 2.0 ** -7), 449.0, 256.0, 447.0, 1.0, 2.0 ** -120, 2.0 ** -133,
                3.3e38, 2.0 ** 127):
        rows.append([top] + [top * f / 64 for f in range(1, d)])
    ties = [1.0625, 1.1875, 17.0, 19.0, 2.0 ** -10, 3 * 2.0 ** -10, -1.0625, -2.0 ** -10, 464.0]
    rows.append([448.0] + ties[:8] + [0.0, -0.0] * 27 + [1.0])
    rows += [[2.0 ** e] * d for e in range(-140, 128, 3)]
    x = torch.tensor(rows, dtype=torch.float64).to(dtype).view(len(rows), 1, d)
    page = 16
    table, pool = table_for([len(rows)], page, 0, 1)
    cache = fa.new_cache(pool, page, 1, d)
    n = torch.tensor([len(rows)], dtype=torch.int32).cuda()
    fa.cache_append(cache, x.cuda(), (-x).cuda(), cu([len(rows)]).cuda(), n, table.cuda(), len(rows))
    host = [t.view(torch.uint8).cpu().numpy() for t in cache]
    for i in range(len(rows)):
        p, r = int(table[0, i // page]), i % page
        for z, s in ((0, 1.0), (1, -1.0)):
            c, e = quantise_row(s * x[i, 0].double().numpy())
            assert (host[z][p, 0, r] == c).all(), (i, z)
            assert host[2 + z][p, 0, r] == e, (i, z)


@gpu
def test_append_and_read_strided_views_equal_contiguous():
    T, Hkv, d, page = 37, 4, 128, 16
    g = torch.Generator().manual_seed(2)
    fused = torch.randn(T, 3 * Hkv, d, generator=g).bfloat16().cuda()
    k, v = fused[:, Hkv:2 * Hkv], fused[:, 2 * Hkv:]
    table, pool = table_for([T], page, 1, 7)
    n, c = torch.tensor([T], dtype=torch.int32).cuda(), cu([T]).cuda()
    a, b = fa.new_cache(pool, page, Hkv, d), fa.new_cache(pool, page, Hkv, d)
    fa.cache_append(a, k, v, c, n, table.cuda(), T)
    fa.cache_append(b, k.contiguous(), v.contiguous(), c, n, table.cuda(), T)
    assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a, b))
    out, whole = guarded_empty((T, 2 * Hkv, d), torch.bfloat16)
    fa.fa_cache_read(a, out[:, :Hkv], out[:, Hkv:], c, table.cuda(), T)
    want = fa.cache_read(a, c, table.cuda(), T, T)
    assert torch.equal(out[:, :Hkv], want[0]) and torch.equal(out[:, Hkv:], want[1])
    whole()
    fa.fa_device_status()


@gpu
def test_bad_tables_and_lengths_touch_nothing_else():
    """Pages outside the pool, positions before 0 or past the table, starts that do not rise and
    rows past the last sequence: dropped on writing, zero on reading, no other byte changes."""
    Hkv, d, page, pool = 2, 64, 16, 6
    guards = []
    tensors = []
    for shape in [(pool, Hkv, page, d)] * 2 + [(pool, Hkv, page)] * 2:
        t, whole = guarded_empty(shape, torch.uint8)
        t.fill_(0x11)
        tensors.append(t)
        guards.append(whole)
    cache = fa.PagedCache(*tensors)
    table = torch.tensor([[0, -1, 2], [pool, 10 ** 9, 3]], dtype=torch.int32)
    x = torch.randn(60, Hkv, d).cuda()
    # sequence 0: positions 38 .. 57 (the last 10 past the table); sequence 1: -5 .. 34
    starts = torch.tensor([0, 20, 60], dtype=torch.int32)
    fa.cache_append(cache, x, x, starts.cuda(),
                    torch.tensor([58, 35], dtype=torch.int32).cuda(), table.cuda(), 40)
    fa.fa_device_status()
    changed = (tensors[0].cpu() != 0x11).any(-1).any(1)  # [pool, page]
    want = torch.zeros(pool, page, dtype=torch.bool)
    want[2, 6:] = True   # positions 38 .. 47 of sequence 0
    want[3, :3] = True   # positions 32 .. 34 of sequence 1
    assert torch.equal(changed, want)
    for whole in guards:
        whole()
    for bad in ([0, 48, 30], [-7, 10, 99], [50, 50, 70]):
        k, kw = guarded_empty((60, Hkv, d), torch.float32)
        v, vw = guarded_empty((60, Hkv, d), torch.float32)
        fa.fa_cache_read(cache, k, v, torch.tensor(bad, dtype=torch.int32).cuda(), table.cuda(), 48)
        fa.fa_device_status()
        kw()
        vw()
    k = torch.full((60, Hkv, d), 7.0).cuda()
    v = k.clone()
    fa.fa_cache_read(cache, k, v, torch.tensor([2, 50, 50], dtype=torch.int32).cuda(), table.cuda(), 48)
    assert (k[:2] == 7).all() and (k[50:] == 7).all()       # no sequence's rows
    assert (k[2 + 16:2 + 32] == 0).all() and (v[2 + 16:2 + 32] == 0).all()  # the missing page


@gpu
def test_append_and_read_under_a_graph():
    Hkv, d, page, B = 4, 128, 64, 3
    lens = [70, 1, 64]
    table, pool = table_for([n + 8 for n in lens], page, 0, 5)
    cache = fa.new_cache(pool, page, Hkv, d)
    k, v = (torch.randn(B, Hkv, d).bfloat16().cuda() for _ in range(2))
    n = torch.tensor(lens, dtype=torch.int32).cuda()
    ones, tab = cu([1] * B).cuda(), table.cuda()
    total = sum(lens) + 4 * B
    out = [torch.zeros(total, Hkv, d, dtype=torch.bfloat16).cuda() for _ in range(2)]
    ends = cu(lens).cuda()
    fa.cache_append(cache, k, v, ones, n, tab, 1)  # the library's first call, before capture
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        n.add_(1)
        ends.add_(torch.arange(B + 1, dtype=torch.int32, device="cuda"))
        fa.cache_append(cache, k, v, ones, n, tab, 1)
        fa.fa_cache_read(cache, out[0], out[1], ends, tab, total)
    for step in range(3):
        k.copy_(torch.randn(k.shape))
        graph.replay()
        torch.cuda.synchronize()
        last = ends[1:].long() - 1
        amax = k.float().abs().amax(-1, keepdim=True)
        assert ((out[0][last].float() - k.float()).abs() <= amax * 2.0 ** -4).all()


# ------------------------------------------------------------------------------ refusals (CPU)

@pytest.fixture(scope="module")
def lib():
    from exact_attention_25_gb300 import _lib, build

    build.build()
    return _lib.load(_lib.LIB_PATH)


BASE = dict(k=0x10000, v=0x20000, st=None, kc=0x30000, vc=0x40000, ke=0x50000, ve=0x60000,
            cu=0x70000, n=0x80000, table=0x90000, B=1, most=4, total=4, max_pages=2, pages=3,
            page=16, Hkv=2, d=64, dtype=0)


def append(lib, a):
    vp = ctypes.c_void_p
    st = None if a["st"] is None else (ctypes.c_longlong * 4)(*a["st"])
    return lib.fa_cache_append(vp(a["k"]), vp(a["v"]), st, vp(a["kc"]), vp(a["vc"]), vp(a["ke"]),
                               vp(a["ve"]), vp(a["cu"]), vp(a["n"]), vp(a["table"]), a["B"],
                               a["most"], a["total"], a["max_pages"], a["pages"], a["page"],
                               a["Hkv"], a["d"], a["dtype"], None)


def read(lib, a):
    vp = ctypes.c_void_p
    st = None if a["st"] is None else (ctypes.c_longlong * 4)(*a["st"])
    return lib.fa_cache_read(vp(a["kc"]), vp(a["vc"]), vp(a["ke"]), vp(a["ve"]), vp(a["k"]),
                             vp(a["v"]), st, vp(a["cu"]), vp(a["table"]), a["B"], a["most"],
                             a["total"], a["max_pages"], a["pages"], a["page"], a["Hkv"], a["d"],
                             a["dtype"], None)


@pytest.mark.parametrize("fn", [append, read])
@pytest.mark.parametrize("kw, code", [
    (dict(dtype=3), -1), (dict(d=32), -2), (dict(B=0), -1), (dict(Hkv=0), -1),
    (dict(max_pages=0), -1), (dict(pages=0), -1), (dict(page=8), -1), (dict(page=48), -1),
    (dict(page=2048), -1), (dict(total=0), -1), (dict(most=0), -1), (dict(k=0), -1),
    (dict(v=0), -1), (dict(kc=0), -1), (dict(ve=0), -1), (dict(table=0), -1), (dict(cu=0), -1),
    (dict(k=0x10008), -3), (dict(vc=0x40004), -3), (dict(ke=0x50008), -3), (dict(cu=0x70001), -3),
    (dict(table=0x90002), -3), (dict(pages=1 << 26, page=16), -7),
    (dict(st=[128, 60, 128, 64]), -3), (dict(st=[128, 32, 128, 64]), -1),
    (dict(st=[64, 128, 128, 64]), -1), (dict(st=[0, 64, 128, 64]), -3),
    (dict(B=1 << 30, most=64, total=64), -7),
])
def test_append_and_read_refuse(lib, fn, kw, code):
    assert fn(lib, {**BASE, **kw}) == code


def test_append_refuses_missing_lengths(lib):
    assert append(lib, {**BASE, "n": 0}) == -1
    assert append(lib, {**BASE, "n": 0x80002}) == -3


def test_binding_checks_the_cache_and_the_integers():
    cache = fa.new_cache(2, 16, 2, 64, device="cpu")
    assert cache.k.shape == (2, 2, 16, 64) and (cache.k_exp == 127).all()
    x = torch.zeros(3, 2, 64)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    tab = torch.zeros(1, 2, dtype=torch.int32)
    with pytest.raises(TypeError):
        fa.cache_append(cache, x, x, i32(0, 3), i32(3), tab.long(), 3)
    with pytest.raises(ValueError):
        fa.cache_append(cache, x, x, i32(0, 3), i32(3), tab, 3)  # not on a CUDA device
    with pytest.raises(ValueError):
        fa.cache_append(cache._replace(k_exp=cache.k_exp[:1]), x, x, i32(0, 3), i32(3), tab, 3)
    with pytest.raises(ValueError):
        fa.cache_append(cache._replace(v=cache.v.float()), x, x, i32(0, 3), i32(3), tab, 3)
