"""What the serving kernels may read, and when.  A kernel launched as a programmatic dependent sees what
the kernels before it wrote only after its own `griddepcontrol.wait`: that its predecessor has waited
orders that kernel's reads, not its own (a cached line of an earlier step's lengths may still lie
beside the SM that it runs on).  A model of that rule, the kernels' sources held to it, and batches
whose lengths grow on the device while units of work are cut between thread blocks."""
import os
import re

import pytest
import torch

import exact_attention_25_gb300 as fa
from tests import test_decode_cache, test_decode_shared
from tests.test_cache import cu, table_for
from tests.test_launch_order import Kernel
from tests.test_serve_protocol import append, host, rope

gpu = pytest.mark.gpu
CSRC = os.path.join(os.path.dirname(fa.__file__), "csrc")


# ------------------------------------------------------------------------------ a model of visibility

def unseen(kernels):
    """Reads of what an earlier kernel wrote by a programmatic dependent that has not waited yet."""
    written, bad = set(), []
    for k in kernels:
        waited = not k.pdl
        for step in k.steps:
            if step[0] == "wait":
                waited = True
            if step[0] == "read" and not waited:
                bad += [(k.name, buf) for buf in step[1:] if buf in written]
        for step in k.steps:
            if step[0] == "write":
                written.update(step[1:])
    return bad


def decode(early):
    """The attention kernel, which leaves the places of the parts, and the merge."""
    att = Kernel("attention", [("wait",), ("trigger",), ("read", "q", "cache", "lens"),
                               ("write", "part", "places", "out")], pdl=True)
    merge = [("wait",), ("trigger",), ("read", "places", "part"), ("write", "out")]
    return [att, Kernel("merge", ([("read", "lens")] if early else []) + merge, pdl=True)]


def step(early=False):
    return [host("producer", (), ("q", "k", "v", "pos", "lens", "table"))] + rope() + append() + decode(early)


def test_a_serving_step_sees_what_was_written_before_it():
    assert unseen(step() + step()) == []


def test_the_model_notices_lengths_read_ahead_of_the_wait():
    assert ("merge", "lens") in unseen(step(early=True))


# ------------------------------------------------------------------------------ the sources

READERS = r"find_share|sequence_work|unit_at|shared_item|shared_places|count_places|packed_rows|cache_row|warp_place"
POINTERS = r"p\.(?:cu\w*|seqlens|table|pos|q|k|v|o|kc|vc|ke|ve|x|y|lse\w*|o_part|cuts|places)\b"


def kernels(name):
    """(kernel, body) of every __global__ function of a source."""
    with open(os.path.join(CSRC, name)) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    for m in re.finditer(r"__global__[^;{]*?(fa_\w+)\s*\([^{;]*\)\s*\{", text):
        depth, at = 1, m.end()
        while depth:
            depth += {"{": 1, "}": -1}.get(text[at], 0)
            at += 1
        yield m.group(1), text[m.end():at]


SOURCES = {"fa_rope.cu": 1, "fa_cache.cu": 2, "fa_decode_cache.cu": 2, "fa_decode_shared.cu": 2}


def test_every_serving_kernel_is_looked_at():
    for name, n in SOURCES.items():
        assert len(list(kernels(name))) == n, name


@pytest.mark.parametrize("name", list(SOURCES))
def test_nothing_is_read_ahead_of_the_wait(name):
    for kernel, body in kernels(name):
        wait = body.index("dependent_begin()")
        early = re.findall(rf"\b(?:{READERS})\s*[(<]|{POINTERS}", body[:wait])
        assert not early, (kernel, early)


# ------------------------------------------------------------------------------ lengths that grow

@gpu
@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("d, H, Hkv, nq", [(128, 8, 2, 1), (64, 16, 2, 3), (128, 4, 4, 2)])
def test_cut_units_of_a_growing_cache(d, H, Hkv, nq, graph):
    """Lengths that a kernel moves on right before the decode, by amounts that move the borders
    between thread blocks through the units; every step against attention in 64 bits over that step's lengths."""
    page, B, ctas, steps = 64, 3, 13, 6
    most, grow = 3200, torch.tensor([131, 517, 260], dtype=torch.int32).cuda()
    table, pool = table_for([most] * B, page, 1, 4)
    codes, exps = test_decode_cache.random_cache(pool, Hkv, page, d, 4)
    cache = test_decode_cache.to_cache(codes, exps)
    tab, starts = table.cuda(), cu([nq] * B).cuda()
    q = torch.randn(B * nq, H, d, generator=torch.Generator().manual_seed(d)).bfloat16().cuda()
    first = torch.tensor([400, 1, 1300], dtype=torch.int32).cuda()
    n = first.clone()
    o, lse = torch.empty_like(q), torch.empty(H, B * nq, device="cuda")
    ws = torch.empty(fa.fa_decode_cache_workspace_bytes(H, Hkv, d, nq, ctas), dtype=torch.uint8).cuda()

    def one():
        n.add_(grow)
        fa.fa_fwd_decode_cache(q, cache, o, lse, starts, n, tab, nq, most, 0.1, True, ctas, ws)

    one()
    n.copy_(first)
    run = one
    if graph:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            one()
        run = g.replay
    got = []
    for _ in range(steps):
        run()
        got.append((n.clone(), o.clone(), lse.clone()))
    torch.cuda.synchronize()
    fa.fa_device_status()
    for i, (lens, a, b) in enumerate(got):
        assert torch.equal(lens, first + (i + 1) * grow)
        ref = test_decode_cache.reference(q.cpu(), codes, exps, table, [nq] * B, lens.tolist(), H, page, 0.1, True)
        test_decode_cache._check((a, b), ref, f"step {i}")


@gpu
@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("d, H, Hkv, nq", [(128, 8, 2, 1), (64, 12, 3, 5), (128, 64, 1, 4)])
def test_cut_units_of_growing_prefixes_and_keys(d, H, Hkv, nq, graph):
    """The same for the decode with shared prefixes: prefixes, own keys and the borders of the groups
    move from step to step; every step against attention in 64 bits."""
    B, ctas, steps, total = 5, 17, 5, 4000
    lens_q = [nq] * B
    x = test_decode_shared.make(lens_q, [total // B] * B, [0, 2, B], [1500, 1500], H, Hkv, d, d + H)
    dev = {n: t.cuda() for n, t in x.items() if n != "sizes"}
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32).cuda()  # noqa: E731
    state = [i32(0, 10, 20, 250, 260, 300), i32(0, 130, 900), i32(0, 1, 5)]     # cu_k, cu_p, cu_g
    grow = [i32(0, 129, 140, 400, 401, 700), i32(0, 270, 390), i32(0, 1, 0)]
    first = [t.clone() for t in state]
    o, lse = torch.empty_like(dev["q"]), torch.empty(H, B * nq, device="cuda")
    ws = torch.empty(fa.fa_decode_shared_workspace_bytes(B * nq, H, d, ctas), dtype=torch.uint8).cuda()

    def one():
        for t, by in zip(state, grow):
            t.add_(by)
        state[2].remainder_(6)
        fa.fa_fwd_decode_shared(dev["q"], dev["kp"], dev["vp"], dev["k"], dev["v"], o, lse, dev["cu_q"], state[0],
                                state[2], state[1], nq, 3000, B * nq, 2000, 0.1, True, ctas, ws)

    one()
    for t, was in zip(state, first):
        t.copy_(was)
    run = one
    if graph:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            one()
        run = g.replay
    got = []
    for _ in range(steps):
        run()
        got.append([t.clone() for t in state + [o, lse]])
    torch.cuda.synchronize()
    fa.fa_device_status()
    for i, (ck, cp, cg, a, b) in enumerate(got):
        part = dict(x, cu_k=ck.cpu(), cu_p=cp.cpu(), cu_g=cg.cpu())
        test_decode_shared.check((a, b), test_decode_shared.reference(part, 0.1, True), f"step {i}")
