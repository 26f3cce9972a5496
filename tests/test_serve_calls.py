"""What a user's program does around the serving calls: tables that are copied and pickled, empty steps,
batches without own keys or prefixes, workspaces that are views, and native bindings that a change of
torch has made stale."""
import copy
import ctypes
import gc
import pickle

import pytest
import torch

import exact_attention_25_gb300 as fa

gpu = pytest.mark.gpu


# ------------------------------------------------------------------------------ copies of a rope table

def behind(table):
    """What lies at the addresses that every call of rope passes."""
    freq, axis = table._args[:2]
    n = table.pairs
    return (tuple((ctypes.c_double * n).from_address(freq)), tuple((ctypes.c_int * n).from_address(axis)))


def _layer():
    m = torch.nn.Module()
    m.table = fa.RopeTable(64, [0.5 ** i for i in range(16)], [0] * 8 + [1] * 8, True)
    return m


@pytest.mark.parametrize("again", [lambda t: copy.deepcopy(t), lambda t: copy.copy(t),
                                   lambda t: pickle.loads(pickle.dumps(t)),
                                   lambda t: copy.deepcopy({"layers": [t, t]})["layers"][1]],
                         ids=["deepcopy", "copy", "pickle", "nested"])
def test_copies_of_a_table_own_what_they_pass(again):
    t = fa.RopeTable(64, [0.5 ** i for i in range(16)], [0] * 8 + [1] * 8, True)
    want, first = (t.inv_freq, t.axis), t._args[:2]
    u = again(t)
    # not the first table's arrays, unless it holds them itself
    assert not set(u._args[:2]) & set(first) or u._freq is t._freq
    del t
    gc.collect()
    # what the allocator would give the arrays' memory to next
    other = [(ctypes.c_double * 16)(*[7.0] * 16) for _ in range(64)]
    assert behind(u) == want == (u.inv_freq, u.axis)
    assert (u.d, u.pairs, u.axes, u.interleaved) == (64, 16, 2, True) and u._args[2:] == (2, 64, 16, True)
    del other


def test_a_copied_module_keeps_its_table():
    m = _layer()
    n = copy.deepcopy(m)
    assert n.table._args[0] != m.table._args[0]
    del m
    gc.collect()
    assert behind(n.table) == (n.table.inv_freq, n.table.axis)


# ------------------------------------------------------------------------------ workspaces that are views

i32 = lambda *v: torch.tensor(v, dtype=torch.int32)  # noqa: E731


@pytest.mark.parametrize("call", ["cache", "shared"])
def test_a_workspace_with_gaps_is_refused(call):
    """The kernels write the workspace as one run of bytes: a view with gaps would have what lies in them
    overwritten."""
    ws = torch.zeros(64, 2, 1024, dtype=torch.uint8)[:, 0]
    assert not ws.is_contiguous()
    q, kv = torch.zeros(2, 4, 64).bfloat16(), torch.zeros(9, 2, 64).bfloat16()
    with pytest.raises(ValueError, match="workspace"):
        if call == "cache":
            fa.fa_fwd_decode_cache(q, fa.new_cache(2, 16, 2, 64, device="cpu"), q.clone(), None, i32(0, 1, 2),
                                   i32(3, 4), torch.zeros(2, 1, dtype=torch.int32), 1, 9, 0.1, False, 2, ws)
        else:
            fa.fa_fwd_decode_shared(q, kv, kv, kv, kv, q.clone(), None, i32(0, 1, 2), i32(0, 4, 9), i32(0, 2),
                                    i32(0, 9), 1, 5, 2, 9, 0.1, False, 2, ws)


# ------------------------------------------------------------------------------ no own keys, no prefixes

@pytest.fixture(scope="module")
def lib():
    from exact_attention_25_gb300 import _lib, build

    build.build()
    return _lib.load(_lib.LIB_PATH)


@pytest.mark.skipif(torch.cuda.is_available(), reason="calls with dummy pointers that pass every check")
@pytest.mark.parametrize("kw", [dict(tk=0, mk=0, k=0, v=0), dict(tp=0, mp=0, kp=0, vp=0), dict(tk=0, mk=0, k=0x60008),
                                dict(tk=0, mk=0, tp=0, mp=0, k=0, v=0, kp=0, vp=0)])
def test_shared_decode_takes_no_own_keys_or_no_prefixes(lib, kw):
    a = dict(q=0x10000, kp=0x20000, vp=0x30000, k=0x40000, v=0x50000, o=0x60000, lse=0x70000, mk=10, mp=100, tk=20,
             tp=100)
    a.update(kw)
    vp = ctypes.c_void_p
    rc = lib.fa_fwd_decode_shared(
        *(vp(a[n]) for n in ("q", "kp", "vp", "k", "v", "o", "lse")), vp(0x90000), vp(0x91000), vp(0x92000),
        vp(0x93000), 2, 1, 1, a["mk"], 2, a["mp"], 2, a["tk"], a["tp"], 4, 2, 64, ctypes.c_float(0.1), 0, 2,
        vp(0xA0000), 1 << 30, None)
    assert rc == -5, lib.fa_last_error()  # every check passed: only the device is missing


@gpu
@pytest.mark.parametrize("most", [0, 7])
@pytest.mark.parametrize("d, H, Hkv", [(64, 4, 1), (128, 16, 8)])
@pytest.mark.parametrize("none", ["own", "prefix", "either"])
def test_shared_decode_of_empty_tensors(none, d, H, Hkv, most):
    """Own keys, prefixes or both are tensors of no rows (`most`: the longest, as the caller has it); or
    tensors with rows of which the longest sequence takes none."""
    from tests import test_decode_shared as t

    lens_q, own, prefix = [1, 3, 2], [5, 130, 40], [300, 17]
    own = [0] * 3 if none != "prefix" else own
    prefix = [0] * 2 if none != "own" else prefix
    x = t.make(lens_q, own, [0, 2, 3], prefix, H, Hkv, d, d, behind=float("nan"))
    if most:
        x.update({n: x[n][:-40] for n in ("k", "v", "kp", "vp")})  # as the sequences have them: perhaps no rows
    mq, mk, mg, mp = x["sizes"]
    x["sizes"] = (mq, mk if any(own) else most, mg, mp if any(prefix) else most)
    for causal in (False, True):
        got = t.run(x, 0.1, causal)
        fa.fa_device_status()
        t.check(got, t.reference(x, 0.1, causal))


# ------------------------------------------------------------------------------ empty steps

@gpu
@pytest.mark.parametrize("rows", [0, 3])
def test_a_step_without_rows_does_nothing(rows):
    """No sequence has a token this step: tensors of no rows, or (rows = 3) padded ones with a longest
    sequence of 0.  Every call returns, writes nothing and reports nothing."""
    H, Hkv, d, page = 4, 2, 64, 16
    rnd = lambda h: torch.randn(rows, h, d).bfloat16().cuda()  # noqa: E731
    q, k, v = rnd(H), rnd(Hkv), rnd(Hkv)
    none, lens = i32(0, 0, 0).cuda(), i32(5, 0).cuda()
    cache = fa.new_cache(4, page, Hkv, d)
    before = [t.view(torch.uint8).clone() for t in cache]
    tab = i32(0, 1).view(2, 1).cuda()
    if rows == 0:
        pos, table = torch.zeros(1, 0, dtype=torch.int32).cuda(), fa.rope_table(d, (32,))
        for f in (fa.rope, fa.rope_backward):
            a, b = f(q, k, pos, table)
            assert a.shape == q.shape and b.shape == k.shape
        assert fa.rope(q, None, pos, table)[1] is None
        fa.fa_rope(q, k, q, k, pos, table)
    fa.cache_append(cache, k, v, none, lens, tab, 0)
    kr, vr = (t.fill_(3.0) for t in fa.cache_read(cache, none, tab, 0, rows))
    assert kr.shape == vr.shape == (rows, Hkv, d)
    fa.fa_cache_read(cache, kr, vr, none, tab, 0)
    o, lse = torch.full_like(q, 3.0), torch.full((H, rows), 4.0, device="cuda")
    out = fa.forward_decode_cache(q, cache, none, lens, tab, 0, 5)
    assert out[0].shape == q.shape and out[1].shape == (H, rows)
    fa.fa_fwd_decode_cache(q, cache, o, lse, none, lens, tab, 0, 5, 0.1, True, 2, None)
    own = torch.randn(5, Hkv, d).bfloat16().cuda()
    a = (own, own, own, own)
    starts = (none, i32(0, 5, 5).cuda(), i32(0, 2).cuda(), i32(0, 5).cuda(), 0, 5, 0, 5)
    out = fa.forward_decode_shared(q, *a, *starts)
    assert out[0].shape == q.shape and out[1].shape == (H, rows)
    fa.fa_fwd_decode_shared(q, *a, o, lse, *starts, 0.1, True, 2, None)
    fa.fa_device_status()
    assert (kr == 3).all() and (vr == 3).all() and (o == 3).all() and (lse == 4).all()
    assert all(torch.equal(t.view(torch.uint8), b) for t, b in zip(cache, before))


@gpu
def test_an_empty_step_is_checked_like_any_other():
    q = torch.zeros(0, 4, 64).bfloat16().cuda()
    cache, ones, tab = fa.new_cache(4, 16, 2, 64), i32(0, 0).cuda(), i32(0).view(1, 1).cuda()
    with pytest.raises(TypeError):
        fa.forward_decode_cache(q.float(), cache, ones, i32(5).cuda(), tab, 0, 5)
    with pytest.raises(ValueError):
        fa.forward_decode_cache(q, cache, ones, i32(5, 5).cuda(), tab, 0, 5)
    with pytest.raises(ValueError):
        fa.rope(q, None, torch.zeros(1, 1, dtype=torch.int32).cuda(), fa.rope_table(64, (32,)))
    with pytest.raises(ValueError):
        fa.cache_append(cache, q, q, ones, i32(5).cuda(), tab, 0)  # 4 heads for a cache of 2


# ------------------------------------------------------------------------------ one long sequence, many short ones

@pytest.mark.skipif(torch.cuda.is_available(), reason="calls with dummy pointers that pass every check")
def test_shared_decode_takes_one_long_and_very_many_short_sequences(lib):
    """The limits go by the queries that there are, not by what every sequence might have."""
    vp = ctypes.c_void_p
    at = [vp((i + 1) << 40) for i in range(11)]
    rc = lib.fa_fwd_decode_shared(*at, 16000, 1, 5000, 5000, 21000, 100, 21000, 21000, 100, 32, 1, 64,
                                  ctypes.c_float(0.1), 0, 152, vp(12 << 40), 1 << 39, None)
    assert rc == -5, lib.fa_last_error()  # only the device is missing


@gpu
def test_shared_decode_of_one_long_and_very_many_short_sequences():
    from tests import test_decode_shared as t

    few, long, H, Hkv, d = 3000, 3000, 256, 2, 64
    g = torch.Generator().manual_seed(3)
    rnd = lambda n, h: torch.randn(n, h, d, generator=g).bfloat16()  # noqa: E731
    q, k, v, kp, vp = rnd(few + long, H), rnd(few + long, Hkv), rnd(few + long, Hkv), rnd(90, Hkv), rnd(90, Hkv)
    starts = torch.cat([torch.arange(few + 1), torch.tensor([few + long])]).to(torch.int32)
    assert (few + 1) * H * long > 2 ** 31
    x = dict(q=q, k=k, v=v, kp=kp, vp=vp, cu_q=starts, cu_k=starts, cu_g=i32(0, few), cu_p=i32(0, 90))
    x["sizes"] = (long, long, few, 90)
    o, lse = t.run(x, 0.1, True)
    fa.fa_device_status()
    heads, rows = [5, 200], list(range(0, few, 7)) + [few - 1]
    part = dict(q=q[rows][:, heads], k=k[rows], v=v[rows], kp=kp, vp=vp, cu_g=i32(0, len(rows)), cu_p=i32(0, 90),
                cu_q=torch.arange(len(rows) + 1, dtype=torch.int32), cu_k=torch.arange(len(rows) + 1, dtype=torch.int32))
    t.check((o[rows][:, heads], lse[heads][:, rows]), t.reference(part, 0.1, True))
    tail = dict(q=q[few:, heads], k=k[few:], v=v[few:], kp=kp, vp=vp, cu_g=i32(1, 1), cu_p=i32(0, 90),
                cu_q=i32(0, long), cu_k=i32(0, long))
    t.check((o[few:, heads], lse[heads, few:]), t.reference(tail, 0.1, True))


# ------------------------------------------------------------------------------ stale native bindings

class _Compiler:
    """subprocess.run that writes the output file and counts."""
    def __init__(self):
        self.calls = 0

    def __call__(self, cmd, **kw):
        self.calls += 1
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("compiled")
        return type("Done", (), dict(returncode=0, stdout="", stderr=""))()


def test_a_binding_of_another_torch_is_built_again(monkeypatch, tmp_path):
    from exact_attention_25_gb300 import build

    run = _Compiler()
    monkeypatch.setattr(build.subprocess, "run", run)
    monkeypatch.setattr(build, "BINDING", str(tmp_path / "_serve.so"))
    monkeypatch.setattr(build, "BUILD", str(tmp_path / "objects"))
    build.build_binding()
    build.build_binding()
    assert run.calls == 1
    monkeypatch.setattr(torch, "__version__", "9.9.9+other")
    build.build_binding()
    build.build_binding()
    assert run.calls == 2
    monkeypatch.setattr(build.sys, "version", "4.0 (other)")
    build.build_binding()
    assert run.calls == 3
    build.build_binding(force=True)
    assert run.calls == 4


def test_a_binding_that_does_not_load_says_so(monkeypatch):
    import builtins

    real = builtins.__import__

    def broken(name, globals=None, locals=None, fromlist=(), level=0):
        if level and "_serve" in (fromlist or ()):
            raise ImportError("undefined symbol: of_another_torch")
        return real(name, globals, locals, fromlist, level)

    fa._native.cache_clear()
    with monkeypatch.context() as m:
        m.setattr(builtins, "__import__", broken)
        with pytest.raises(ImportError, match="of_another_torch.*build_all"):
            fa._native()
    assert fa._native().rope


# ------------------------------------------------------------------------------ integers inside the outputs

@pytest.mark.parametrize("name", ["cu", "n", "table"])
@pytest.mark.parametrize("at", [0x30000, 0x41000, 0x50000, 0x60020])
def test_append_refuses_integers_inside_the_cache(lib, name, at):
    from tests import test_cache

    assert test_cache.append(lib, {**test_cache.BASE, name: at}) == -1
    assert b"overlap" in lib.fa_last_error()


@pytest.mark.parametrize("name", ["cu", "table"])
@pytest.mark.parametrize("at", [0x10000, 0x20100])
def test_read_refuses_integers_inside_its_outputs(lib, name, at):
    from tests import test_cache

    assert test_cache.read(lib, {**test_cache.BASE, name: at}) == -1
    assert b"overlap" in lib.fa_last_error()


# ------------------------------------------------------------------------------ calls without lse, long pages

@gpu
@pytest.mark.parametrize("ctas", [1, 7])
def test_decodes_without_lse_give_the_same_outputs(ctas):
    from tests import test_decode_cache as c
    from tests import test_decode_shared as t
    from tests.test_cache import cu, table_for

    H, Hkv, d, page, lens_q, lens_k = 8, 2, 128, 64, [1, 2], [700, 90]
    table, pool = table_for(lens_k, page, 1, 3)
    cache = c.to_cache(*c.random_cache(pool, Hkv, page, d, 3))
    q = torch.randn(3, H, d, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    a = (cu(lens_q).cuda(), i32(*lens_k).cuda(), table.cuda(), 2, 700, 0.1, True, ctas)
    want = fa.forward_decode_cache(q, cache, *a)
    o = torch.empty_like(q)
    ws = torch.empty(max(fa.fa_decode_cache_workspace_bytes(H, Hkv, d, 2, ctas), 16), dtype=torch.uint8).cuda()
    fa.fa_fwd_decode_cache(q, cache, o, None, *a, ws)
    assert torch.equal(o, want[0])
    x = t.make([1, 2, 1], [30, 200, 5], [0, 3], [900], H, Hkv, d, 2)
    dev = {n: v.cuda() for n, v in x.items() if n != "sizes"}
    want = t.run(x, 0.1, True, ctas)
    o = torch.empty_like(dev["q"])
    ws = torch.empty(fa.fa_decode_shared_workspace_bytes(4, H, d, ctas), dtype=torch.uint8).cuda()
    fa.fa_fwd_decode_shared(*(dev[n] for n in ("q", "kp", "vp", "k", "v")), o, None,
                            *(dev[n] for n in ("cu_q", "cu_k", "cu_g", "cu_p")), *x["sizes"], 0.1, True, ctas, ws)
    assert torch.equal(o, want[0])
    fa.fa_device_status()


@gpu
@pytest.mark.parametrize("ctas", [None, 5])
@pytest.mark.parametrize("page", [256, 512, 1024])
def test_cache_decode_over_long_pages(page, ctas):
    from tests import test_decode_cache as c

    c.run_case([1, 4, 2], [2500, 1024, 7], 8, 2, 64, page, True, ctas, seed=page)
    c.run_case([1, 1], [1025, 513], 4, 4, 128, page, False, ctas, seed=page + 1)
