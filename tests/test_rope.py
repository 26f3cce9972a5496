"""Rotary positions with several axes (fa_rope): against angles reduced in 60 digits, both pair
layouts and types, partial rotation, far and negative positions, strided and in-place calls; the
backward against the formula, differences and the forward's inverse; refusals."""
import ctypes

import numpy as np
import pytest
import torch

import exact_attention_25_gb300 as fa
from tests.gpu_util import guarded_empty
from tests.serve_util import HALF_STEP, rope_reference

gpu = pytest.mark.gpu


def make(total, H, Hkv, d, axes, dtype, seed, far=100000):
    g = torch.Generator().manual_seed(seed)
    q = torch.randn(total, H, d, generator=g).to(dtype)
    k = torch.randn(total, Hkv, d, generator=g).to(dtype) if Hkv else None
    pos = torch.randint(-far, far, (axes, total), generator=g, dtype=torch.int32)
    return q, k, pos


def check(got, x, pos, table, inverse, dtype):
    """Bounds: sine and cosine are off by at most 2^-24 (the function) + pi/4 * 2^-24 (its
    argument in fp32) + 2^-30 (the fixed-point angle), the two products and their sum by 2 * 2^-24
    of |x1| + |x2|; in all below 2^-22 (|x1| + |x2|), then half a step of the type."""
    x64 = x.double().numpy()
    ref = rope_reference(x64, pos.numpy(), table.inv_freq, table.axis, table.interleaved, inverse)
    n = table.pairs
    size = np.zeros_like(x64)
    for p in range(n):
        i, j = (2 * p, 2 * p + 1) if table.interleaved else (p, n + p)
        size[..., i] = size[..., j] = np.abs(x64[..., i]) + np.abs(x64[..., j])
    err = np.abs(got.double().cpu().numpy() - ref)
    tol = HALF_STEP[dtype] * np.abs(ref) * (1 + 2.0 ** -20) + 2.0 ** -22 * size
    assert (err <= tol).all(), float((err / np.maximum(tol, 1e-300)).max())
    assert torch.equal(got[..., 2 * n:].cpu(), x[..., 2 * n:])  # what is not turned is copied


CASES = {
    # name: (tokens, H, Hkv, d, sections, per_axis, interleaved, dtype)
    "one_token": (1, 4, 1, 128, (16, 24, 24), False, False, torch.bfloat16),
    "gqa_fp32": (5, 7, 2, 64, (16, 16), True, True, torch.float32),
    "mqa_interleaved": (33, 16, 1, 128, (64,), False, True, torch.bfloat16),
    "partial": (17, 3, 3, 128, (5, 11, 16), False, False, torch.float32),
    "partial_interleaved": (9, 2, 1, 64, (3, 5), True, True, torch.bfloat16),
    "four_axes": (40, 32, 8, 128, (1, 30, 2, 31), True, False, torch.bfloat16),
    "q_only": (6, 5, 0, 64, (32,), False, False, torch.bfloat16),
    "many_tokens": (3001, 2, 1, 64, (8, 24), False, False, torch.bfloat16),
}


@gpu
@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("case", list(CASES))
def test_rope_against_the_definition(case, inverse):
    total, H, Hkv, d, sections, per_axis, inter, dtype = CASES[case]
    table = fa.rope_table(d, sections, 10000.0, per_axis, inter)
    q, k, pos = make(total, H, Hkv, d, len(sections), dtype, seed=len(case))
    call = fa.rope_backward if inverse else fa.rope
    qo, ko = call(q.cuda(), None if k is None else k.cuda(), pos.cuda(), table)
    check(qo, q, pos, table, inverse, dtype)
    if k is None:
        assert ko is None
    else:
        check(ko, k, pos, table, inverse, dtype)


@gpu
def test_rope_of_the_farthest_positions_keeps_the_angle():
    """Positions at the ends of int32, whose angles lose all 24 bits of an fp32 product."""
    table = fa.rope_table(128, (64,), 500000.0)
    q, k, pos = make(6, 2, 1, 128, 1, torch.float32, 3)
    pos[0] = torch.tensor([2 ** 31 - 1, -2 ** 31, 2 ** 30 + 12345, 0, -1, 16777217])
    qo, ko = fa.rope(q.cuda(), k.cuda(), pos.cuda(), table)
    check(qo, q, pos, table, False, torch.float32)
    check(ko, k, pos, table, False, torch.float32)


@gpu
def test_rope_with_given_frequencies_and_axes():
    """Frequencies outside (0, 1], negative ones and axes in any order."""
    g = torch.Generator().manual_seed(5)
    freq = (torch.rand(32, generator=g, dtype=torch.float64) * 20 - 10).tolist()
    freq[:3] = [0.0, 1048576.0, -1e-12]
    axis = torch.randint(0, 3, (32,), generator=g).tolist()
    table = fa.RopeTable(64, freq, axis, True)
    q, k, pos = make(21, 3, 1, 64, 3, torch.float32, 4)
    qo, ko = fa.rope(q.cuda(), k.cuda(), pos.cuda(), table)
    check(qo, q, pos, table, False, torch.float32)
    check(ko, k, pos, table, False, torch.float32)


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rope_strided_views_in_place_and_guards(dtype):
    """q and k as views of one fused projection, turned into other views and in place; equal to
    the contiguous call bit for bit, and nothing else is written."""
    total, H, Hkv, d = 19, 6, 2, 128
    table = fa.rope_table(d, (16, 24, 24))
    g = torch.Generator().manual_seed(1)
    fused = torch.randn(total, H + 2 * Hkv, d, generator=g).to(dtype).cuda()
    pos = torch.randint(0, 5000, (3, total), generator=g, dtype=torch.int32).cuda()
    q, k = fused[:, :H], fused[:, H:H + Hkv]
    want_q, want_k = fa.rope(q.contiguous(), k.contiguous(), pos, table)
    out, whole = guarded_empty((total, H + 2 * Hkv, d), dtype)
    fa.fa_rope(q, k, out[:, :H], out[:, H:H + Hkv], pos, table)
    assert torch.equal(out[:, :H], want_q) and torch.equal(out[:, H:H + Hkv], want_k)
    assert (out[:, H + Hkv:] == 0).all()
    whole()
    before = fused[:, H + Hkv:].clone()
    fa.fa_rope(q, k, q, k, pos, table)
    assert torch.equal(q, want_q) and torch.equal(k, want_k)
    assert torch.equal(fused[:, H + Hkv:], before)
    fa.fa_device_status()


@gpu
def test_rope_backward_is_the_gradient():
    """Of L = sum(w * rope(x)): against differences of the forward in fp32 (the map is linear, so
    the difference quotient is exact up to rounding), and turning there and back."""
    total, H, d = 4, 2, 64
    table = fa.rope_table(d, (10, 22), 1000.0, True, True)
    q, _, pos = make(total, H, 0, d, 2, torch.float32, 9, far=500)
    w = torch.randn(q.shape, generator=torch.Generator().manual_seed(2))
    dq, _ = fa.rope_backward(w.cuda(), None, pos.cuda(), table)
    for at in [(0, 0, 0), (1, 1, 7), (3, 0, 63), (2, 1, 32)]:
        e = torch.zeros_like(q)
        e[at] = 1.0
        y, _ = fa.rope(e.cuda(), None, pos.cuda(), table)
        want = float((y.cpu().double() * w.double()).sum())
        # two products of unit size, each side good to 2^-22 of |w1| + |w2|
        assert abs(float(dq[at]) - want) <= 2.0 ** -21 * 2 * float(w.abs().max())
    there, _ = fa.rope(q.cuda(), None, pos.cuda(), table)
    back, _ = fa.rope_backward(there, None, pos.cuda(), table)
    assert (back.cpu() - q).abs().max() <= 2.0 ** -21 * 2 * 2 * q.abs().max()


@gpu
def test_rope_under_a_graph_and_on_another_stream():
    table = fa.rope_table(128, (16, 24, 24))
    q, k, pos = (t.cuda() for t in make(50, 8, 2, 128, 3, torch.bfloat16, 11))
    want = fa.rope(q, k, pos, table)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = fa.rope(q, k, pos, table, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fa.fa_rope(q, k, qo, ko, pos, table)
    for _ in range(2):
        q.copy_(torch.randn(q.shape).to(q.dtype))
        pos.add_(17)
        graph.replay()
        want = fa.rope(q, k, pos, table)
        assert torch.equal(qo, want[0]) and torch.equal(ko, want[1])


# ------------------------------------------------------------------------------ refusals (CPU)

@pytest.fixture(scope="module")
def lib():
    from exact_attention_25_gb300 import _lib, build

    build.build()
    return _lib.load(_lib.LIB_PATH)


def call(lib, **kw):
    a = dict(q=0x10000, k=0x20000, qo=0x30000, ko=0x40000, pos=0x50000, freq=[0.5] * 32,
             axis=[0] * 32, strides=None, total=2, H=2, Hkv=1, d=64, axes=1, pairs=32, inter=0,
             inverse=0, dtype=0)
    a.update(kw)
    vp = ctypes.c_void_p
    freq = None if a["freq"] is None else (ctypes.c_double * 64)(*a["freq"])
    axis = None if a["axis"] is None else (ctypes.c_int * 64)(*a["axis"])
    st = None if a["strides"] is None else (ctypes.c_longlong * 8)(*a["strides"])
    return lib.fa_rope(vp(a["q"]), vp(a["k"]), vp(a["qo"]), vp(a["ko"]), vp(a["pos"]), freq, axis,
                       st, a["total"], a["H"], a["Hkv"], a["d"], a["axes"], a["pairs"],
                       a["inter"], a["inverse"], a["dtype"], None)


@pytest.mark.parametrize("kw, code", [
    (dict(dtype=2), -1), (dict(total=0), -1), (dict(H=0), -1), (dict(Hkv=-1), -1),
    (dict(d=96), -2), (dict(axes=0), -1), (dict(axes=9), -1), (dict(pairs=0), -1),
    (dict(pairs=12), -1), (dict(pairs=40), -1), (dict(inter=2), -1), (dict(inverse=-1), -1),
    (dict(q=0), -1), (dict(k=0), -1), (dict(ko=0), -1), (dict(pos=0), -1), (dict(freq=None), -1),
    (dict(axis=None), -1), (dict(axis=[1] * 32), -1), (dict(axis=[-1] * 32), -1),
    (dict(freq=[float("nan")] * 32), -1), (dict(freq=[float("inf")] * 32), -1),
    (dict(freq=[2e6] * 32), -1), (dict(q=0x10008), -3), (dict(ko=0x40004), -3),
    (dict(pos=0x50002), -3), (dict(qo=0x10010), -1), (dict(ko=0x30000), -1),
    (dict(qo=0x20000), -1), (dict(qo=0x50000), -1),
    (dict(strides=[128, 64, 64, 64, 128, 60, 64, 64]), -3),
    (dict(strides=[128, 64, 64, 64, 64, 128, 64, 64]), -1),
    (dict(strides=[128, 32, 64, 64, 128, 64, 64, 64]), -1),
    (dict(total=2 ** 30, H=128, pos=0x500000000000), -7),
])
def test_rope_refuses(lib, kw, code):
    assert call(lib, **kw) == code


def test_rope_binding_refuses():
    q = torch.zeros(4, 2, 64)
    pos = torch.zeros(1, 4, dtype=torch.int32)
    table = fa.rope_table(64, (32,))
    with pytest.raises(ValueError):
        fa.rope(q, None, pos, table)  # not on a CUDA device
    with pytest.raises(ValueError):
        fa.RopeTable(64, [1.0] * 8, [0] * 7)


def test_rope_table_conventions():
    t = fa.rope_table(128, (16, 24, 24))
    assert t.pairs == 64 and t.axes == 3 and t.axis == (0,) * 16 + (1,) * 24 + (2,) * 24
    assert t.inv_freq[0] == 1.0 and abs(t.inv_freq[32] - 0.01) < 1e-15
    t = fa.rope_table(64, (16, 16), 10000.0, True)
    assert t.inv_freq[:16] == t.inv_freq[16:] and abs(t.inv_freq[8] - 0.01) < 1e-15
