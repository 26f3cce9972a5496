"""What the serving-side operators are measured on: rotary positions with several axes, the e4m3
paged key/value cache (append, read back), split-KV decoding over that cache, and decoding of
batches whose sequences share long prefixes.

``run`` computes each operator either in plain torch operations (``own`` false) or by the calls a
user makes of ``exact_attention_25_gb300`` (``own`` true), on the same state.
"""
import math
import random

import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------------------------- cases

def listed():
    return [
        # one decoding step of 8 sequences: the queries and keys of 8 tokens with (time, height,
        # width) positions
        dict(name="rope_step_8", op="rope", tokens=8, H=32, Hkv=8, d=128, sections="16,24,24",
             per_axis=False, interleaved=False, base=10000.0, far=32768, dtype="bf16",
             inverse=False),
        # prefill of one 32000-token sequence of video, full multi-head
        dict(name="rope_video_32000", op="rope", tokens=32000, H=32, Hkv=32, d=128,
             sections="16,24,24", per_axis=False, interleaved=False, base=10000.0, far=32000,
             dtype="bf16", inverse=False),
        # a training step's gradients of 4 images of a little over 4096 patches (height, width),
        # fp32, adjacent pairs, frequencies starting afresh for each axis
        dict(name="rope_bwd_image_fp32", op="rope", tokens=4 * 4097, H=16, Hkv=16, d=64,
             sections="16,16", per_axis=True, interleaved=True, base=10000.0, far=1000,
             dtype="fp32", inverse=True),
        # one new token of each of 64 sequences goes into the cache
        dict(name="append_step_64", op="append", B=64, new=1, new_min=1, hist=1000, Hkv=8, d=128,
             page=64, dtype="bf16", ragged=1),
        # ragged prompts go into the cache, behind histories that end inside a page
        dict(name="append_prompts", op="append", B=9, new=8192, new_min=1, hist=100, Hkv=8, d=128,
             page=64, dtype="bf16", ragged=2),
        # a short history is read back for a chunk of prefill
        dict(name="read_1000", op="read", B=1, hist=1000, hist_min=1000, Hkv=8, d=128, page=16,
             dtype="bf16", ragged=3),
        # 8 ragged histories of up to 16 K keys are read back
        dict(name="read_8x16k", op="read", B=8, hist=16384, hist_min=1, Hkv=8, d=128, page=64,
             dtype="bf16", ragged=4),
        # one token of one sequence over a 4 K history: latency
        dict(name="decode_1x4k", op="decode", B=1, nq=1, nq_min=1, hist=4096, hist_min=4096, H=32,
             Hkv=8, d=128, page=64, causal=True, ragged=5),
        # a serving step: 8 sequences of up to 32 K keys
        dict(name="decode_8x32k", op="decode", B=8, nq=1, nq_min=1, hist=32768, hist_min=3000,
             H=32, Hkv=8, d=128, page=64, causal=True, ragged=6),
        # speculative decoding, up to 4 queries a sequence, small heads, small pages
        dict(name="decode_spec_16x5000", op="decode", B=16, nq=4, nq_min=1, hist=5000, hist_min=0,
             H=16, Hkv=2, d=64, page=16, causal=True, ragged=7),
        # 8 continuations of one 4 K prompt
        dict(name="shared_8x4k", op="shared", groups=1, B=8, nq=1, nq_min=1, prefix=4096,
             prefix_min=4096, hist=257, hist_min=1, H=32, Hkv=8, d=128, causal=True, ragged=8),
        # 64 sequences over a 32000-token prompt, with up to 1024 keys of their own
        dict(name="shared_64x32k", op="shared", groups=1, B=64, nq=1, nq_min=1, prefix=32000,
             prefix_min=32000, hist=1024, hist_min=1, H=32, Hkv=8, d=128, causal=True, ragged=9),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "append", "read", "decode", "shared"])
    d = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 4, 7, 8, 16])
    ragged = rng.randrange(1 << 20)
    page = rng.choice([16, 32, 64, 128])
    if op == "rope":
        axes = rng.choice([1, 2, 3, 4])
        pairs = rng.choice([d // 2, d // 2, d // 4])
        cuts = sorted(rng.sample(range(1, pairs), axes - 1))
        sections = [b - a for a, b in zip([0] + cuts, cuts + [pairs])]
        H = G * Hkv if G * Hkv <= 64 else 32
        return dict(op=op, tokens=min(_log(rng, 1, 32000), 130000000 // ((H + Hkv) * d)), H=H,
                    Hkv=Hkv, d=d, sections=",".join(map(str, sections)),
                    per_axis=rng.random() < 0.5, interleaved=rng.random() < 0.5,
                    base=rng.choice([10000.0, 500000.0, 1e6]), far=_log(rng, 100, 1 << 20),
                    dtype=rng.choice(["bf16", "fp32"]), inverse=rng.random() < 0.5)
    if op == "append":
        B, new = _log(rng, 1, 96), _log(rng, 1, 4000)
        new = min(new, max(1, 60000 // B))
        return dict(op=op, B=B, new=new, new_min=rng.choice([0, 1]), hist=_log(rng, 1, 500),
                    Hkv=Hkv, d=d, page=page, dtype=rng.choice(["bf16", "fp32"]), ragged=ragged)
    if op == "read":
        B = _log(rng, 1, 64)
        return dict(op=op, B=B, hist=_log(rng, 1, 100000 // B), hist_min=0, Hkv=Hkv, d=d,
                    page=page, dtype=rng.choice(["bf16", "fp32"]), ragged=ragged)
    if op == "decode":
        B = _log(rng, 1, 64)
        nq = rng.choice([1, 1, 2, 3, 8]) if G * Hkv <= 32 else rng.choice([1, 1, 2])
        return dict(op=op, B=B, nq=nq, nq_min=rng.choice([0, 1]), hist=_log(rng, 1, 200000 // B),
                    hist_min=rng.choice([0, 1]), H=G * Hkv, Hkv=Hkv, d=d, page=page,
                    causal=rng.random() < 0.7, ragged=ragged)
    groups = rng.choice([1, 1, 2, 3])
    B, nq = _log(rng, groups, 64), rng.choice([1, 1, 2, 4])
    most = min(32000, 60000000 // (B * nq * G * Hkv))
    return dict(op=op, groups=groups, B=B, nq=nq, nq_min=rng.choice([0, 1]),
                prefix=_log(rng, 1, most), prefix_min=1,
                hist=_log(rng, 1, 1500), hist_min=rng.choice([0, 1]), H=G * Hkv, Hkv=Hkv, d=d,
                causal=rng.random() < 0.7, ragged=ragged)


def _spread(rng, n, lo, hi):
    """n lengths in [lo, hi], the first of them hi."""
    return [hi] + [rng.randint(min(lo, hi), hi) for _ in range(n - 1)]


def _lengths(c):
    """The sequence lengths of a case: new tokens or queries, keys in the cache (or of a
    sequence's own), and the prefixes and sizes of the groups."""
    rng = random.Random(c["ragged"])
    B = c["B"]
    if c["op"] == "append":
        new = _spread(rng, B, c["new_min"], c["new"])
        return dict(new=new, keys=[n + rng.randint(0, c["hist"]) for n in new])
    if c["op"] == "read":
        return dict(keys=_spread(rng, B, c["hist_min"], c["hist"]))
    out = dict(keys=_spread(rng, B, c["hist_min"], c["hist"]),
               new=_spread(rng, B, c["nq_min"], c["nq"]))
    if c["op"] == "shared":
        g = c["groups"]
        cuts = sorted(rng.sample(range(1, B), g - 1)) if g > 1 else []
        out["group"] = [0] + cuts + [B]
        out["prefix"] = _spread(rng, g, c["prefix_min"], c["prefix"])
    return out


def work(c):
    es = 4 if c.get("dtype") == "fp32" else 2
    if c["op"] == "rope":
        n = c["tokens"] * (c["H"] + c["Hkv"]) * c["d"]
        axes = c["sections"].count(",") + 1
        return {"bytes": 2 * n * es + 4 * axes * c["tokens"], "flops": 3 * n}
    L = _lengths(c)
    row = c["Hkv"] * c["d"]
    if c["op"] in ("append", "read"):
        n = sum(L["new"] if c["op"] == "append" else L["keys"])
        return {"bytes": 2 * n * (row * (es + 1) + c["Hkv"]), "flops": 2 * n * row}
    tok = sum(L["new"])
    pairs = sum(n * k for n, k in zip(L["new"], L["keys"]))
    io = tok * c["H"] * (4 * c["d"] + 4)  # q and o in bf16, lse in fp32
    if c["op"] == "decode":
        keys = sum(k for n, k in zip(L["new"], L["keys"]) if n)
        return {"bytes": io + 2 * keys * (row + c["Hkv"]), "flops": 4 * c["H"] * c["d"] * pairs}
    keys = sum(k for n, k in zip(L["new"], L["keys"]) if n)
    for g, np_ in enumerate(L["prefix"]):
        t = sum(L["new"][L["group"][g]:L["group"][g + 1]])
        keys += np_ if t else 0
        pairs += np_ * t
    return {"bytes": io + 4 * keys * row, "flops": 4 * c["H"] * c["d"] * pairs}


# ------------------------------------------------------------------------------------ inputs

def _starts(lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return torch.tensor(out, dtype=torch.int32, device=DEV)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _normal(gen, *shape, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=gen, device=DEV, dtype=torch.float32).to(dtype)


def _rows(gen, n, heads, d, dtype=torch.bfloat16):
    """Key or value rows: normal values whose size differs from row to row and from channel to
    channel, as activations' do."""
    x = torch.randn(n, heads, d, generator=gen, device=DEV)
    x *= torch.exp(0.5 * torch.randn(n, heads, 1, generator=gen, device=DEV))
    x *= torch.exp(0.25 * torch.randn(1, heads, d, generator=gen, device=DEV))
    return x.to(dtype)


def _codes(x):
    """Rows in e4m3 with a power-of-two scale a row: (codes, biased exponents)."""
    x = x.float()
    size = torch.where(torch.isfinite(x), x.abs(), torch.zeros_like(x)).amax(-1)
    m, e = torch.frexp(size)  # size = m 2^e, 0.5 <= m < 1
    e = torch.where(m > 0.875, e - 8, e - 9).clamp(-110, 120)
    e = torch.where(size > 0, e, torch.zeros_like(e))
    x = torch.where(torch.isfinite(x), x, torch.full_like(x, float("nan")))
    y = x * torch.exp2(-e.float()).unsqueeze(-1)
    return y.to(torch.float8_e4m3fn), (e + 127).to(torch.uint8)


def _paged(gen, c, keys, fill):
    """Pages for `keys` cached tokens a sequence, in random order in a pool with some to spare;
    fill: with codes of random rows, else zero."""
    need = [-(-n // c["page"]) for n in keys]
    pool = sum(need) + 3
    order = torch.randperm(pool, generator=gen, device=DEV).to(torch.int32)
    table = torch.zeros(len(keys), max(max(need), 1), dtype=torch.int32, device=DEV)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    shape = (pool, c["Hkv"], c["page"], c["d"])
    if fill:
        made = [_codes(_rows(gen, pool * c["page"], c["Hkv"], c["d"]).view(
            pool, c["page"], c["Hkv"], c["d"]).transpose(1, 2)) for _ in range(2)]
        cache = tuple(m[0].contiguous() for m in made) + tuple(m[1].contiguous() for m in made)
    else:
        cache = tuple(torch.zeros(shape, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
                      for _ in range(2))
        cache += tuple(torch.full(shape[:3], 127, dtype=torch.uint8, device=DEV) for _ in range(2))
    return cache, table


def prepare(c, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    s = dict(c)
    dt = torch.float32 if c.get("dtype") == "fp32" else torch.bfloat16
    if c["op"] == "rope":
        sections = tuple(int(x) for x in c["sections"].split(","))
        s["sections"] = sections
        s["q"] = _normal(gen, c["tokens"], c["H"], c["d"], dtype=dt)
        s["k"] = _normal(gen, c["tokens"], c["Hkv"], c["d"], dtype=dt)
        s["pos"] = torch.randint(0, c["far"], (len(sections), c["tokens"]), generator=gen,
                                 device=DEV, dtype=torch.int32)
        return s
    L = _lengths(c)
    s["max_k"] = max(max(L["keys"]), 1)
    s["scale"] = c["d"] ** -0.5
    if c["op"] == "append":
        s["max_new"] = max(L["new"])
        s["cu_new"], s["seqlens"] = _starts(L["new"]), _ints(L["keys"])
        s["cache"], s["table"] = _paged(gen, c, L["keys"], False)
        s["k"], s["v"] = (_rows(gen, sum(L["new"]), c["Hkv"], c["d"], dt) for _ in range(2))
        return s
    if c["op"] == "read":
        s["cu_k"], s["total_k"] = _starts(L["keys"]), sum(L["keys"])
        s["cache"], s["table"] = _paged(gen, c, L["keys"], True)
        s["out_dtype"] = dt
        return s
    tokens = sum(L["new"])
    s["max_q"] = max(L["new"])
    s["cu_q"] = _starts(L["new"])
    s["q"] = _normal(gen, tokens, c["H"], c["d"])
    if c["op"] == "decode":
        s["seqlens"] = _ints(L["keys"])
        s["cache"], s["table"] = _paged(gen, c, L["keys"], True)
        return s
    s["cu_k"], s["cu_p"], s["cu_g"] = _starts(L["keys"]), _starts(L["prefix"]), _ints(L["group"])
    s["max_p"] = max(L["prefix"])
    s["max_group"] = max(sum(L["new"][a:b]) for a, b in zip(L["group"], L["group"][1:]))
    own_keys = max(sum(L["keys"]), 1)
    s["k"], s["v"] = (_normal(gen, own_keys, c["Hkv"], c["d"]) for _ in range(2))
    s["kp"], s["vp"] = (_normal(gen, sum(L["prefix"]), c["Hkv"], c["d"]) for _ in range(2))
    return s


# --------------------------------------------------------------------------------------- run

def run(s):
    return _own(s) if own else _PLAIN[s["op"]](s)


def _own(s):
    import exact_attention_25_gb300 as fa

    if s["op"] == "rope":
        table = fa.rope_table(s["d"], s["sections"], s["base"], s["per_axis"], s["interleaved"])
        call = fa.rope_backward if s["inverse"] else fa.rope
        return call(s["q"], s["k"], s["pos"], table)
    if s["op"] == "shared":
        return fa.forward_decode_shared(
            s["q"], s["kp"], s["vp"], s["k"], s["v"], s["cu_q"], s["cu_k"], s["cu_g"], s["cu_p"],
            s["max_q"], s["max_k"], s["max_group"], s["max_p"], s["scale"], s["causal"])
    cache = fa.PagedCache(*s["cache"])
    if s["op"] == "append":
        fa.cache_append(cache, s["k"], s["v"], s["cu_new"], s["seqlens"], s["table"], s["max_new"])
        return s["cache"]
    if s["op"] == "read":
        return fa.cache_read(cache, s["cu_k"], s["table"], s["max_k"], s["total_k"],
                             s["out_dtype"])
    return fa.forward_decode_cache(s["q"], cache, s["cu_q"], s["seqlens"], s["table"], s["max_q"],
                                   s["max_k"], s["scale"], s["causal"])


def _frequencies(d, sections, base, per_axis):
    """(inverse frequency, axis) of every rotated pair: one run of frequencies over the rotated
    part of the head, or one for each axis."""
    pairs = sum(sections)
    freq, axis = [], []
    for a, n in enumerate(sections):
        for i in range(n):
            freq.append(base ** (-i / n) if per_axis else base ** (-len(freq) / pairs))
            axis.append(a)
    return freq, axis


def _plain_rope(s):
    freq, axis = _frequencies(s["d"], s["sections"], s["base"], s["per_axis"])
    pairs = len(freq)
    # far positions times a frequency need more than 24 bits for the angle's fraction
    angle = (s["pos"].double()[torch.tensor(axis, device=DEV)]
             * torch.tensor(freq, dtype=torch.float64, device=DEV).unsqueeze(1)).t().unsqueeze(1)
    cos, sin = angle.cos().float(), angle.sin().float()
    if s["inverse"]:
        sin = -sin

    def turned(x):
        y = x.float()
        if s["interleaved"]:
            a, b = y[..., 0:2 * pairs:2], y[..., 1:2 * pairs:2]
            z = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
        else:
            a, b = y[..., :pairs], y[..., pairs:2 * pairs]
            z = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
        return torch.cat((z, y[..., 2 * pairs:]), -1).to(x.dtype)

    return turned(s["q"]), turned(s["k"])


def _owners(cu, n):
    """(sequence, index within it) of each of n packed rows."""
    rows = torch.arange(n, device=DEV)
    b = torch.searchsorted(cu[1:].long(), rows, right=True)
    return b, rows - cu.long()[b]


def _plain_append(s):
    b, i = _owners(s["cu_new"], s["k"].shape[0])
    at = s["seqlens"].long()[b] - (s["cu_new"][1:] - s["cu_new"][:-1]).long()[b] + i
    page, off = s["table"].long()[b, at // s["page"]], at % s["page"]
    kc, vc, ke, ve = s["cache"]
    k, v = _codes(s["k"]), _codes(s["v"])
    kc.view(torch.uint8)[page, :, off] = k[0].view(torch.uint8)
    vc.view(torch.uint8)[page, :, off] = v[0].view(torch.uint8)
    ke[page, :, off] = k[1]
    ve[page, :, off] = v[1]
    return s["cache"]


def _values(codes, exps):
    return codes.float() * torch.exp2(exps.float() - 127.0).unsqueeze(-1)


def _plain_read(s):
    b, i = _owners(s["cu_k"], s["total_k"])
    page, off = s["table"].long()[b, i // s["page"]], i % s["page"]
    kc, vc, ke, ve = s["cache"]
    k = _values(kc.view(torch.uint8)[page, :, off].view(torch.float8_e4m3fn), ke[page, :, off])
    v = _values(vc.view(torch.uint8)[page, :, off].view(torch.float8_e4m3fn), ve[page, :, off])
    return k.to(s["out_dtype"]), v.to(s["out_dtype"])


def _padded(x, cu, most):
    """Packed rows as [sequences, most, ...] (rows past a sequence's end repeat some row), and
    the lengths."""
    lens = (cu[1:] - cu[:-1]).long()
    at = cu[:-1].long().unsqueeze(1) + torch.arange(max(most, 1), device=DEV)
    return x[at.clamp(max=x.shape[0] - 1)], lens


def _softmax_parts(q, k, v, seen, scale):
    """q [B, n, H, d], k, v [B, L, Hkv, d] in fp32, seen [B, n, L]: the running maximum, the sum
    and the unnormalised output of each query, [B, n, H(, d)]."""
    B, n, H, d = q.shape
    Hkv = k.shape[2]
    G = H // Hkv
    rows = q.view(B, n, Hkv, G, d).permute(0, 2, 1, 3, 4).reshape(B, Hkv, n * G, d)
    x = torch.matmul(rows, k.permute(0, 2, 3, 1)) * scale
    x = x.view(B, Hkv, n, G, -1).masked_fill(~seen[:, None, :, None, :], -math.inf)
    m = x.amax(-1)
    p = torch.exp(x - m.masked_fill(m == -math.inf, 0.0).unsqueeze(-1))
    acc = torch.matmul(p.view(B, Hkv, n * G, -1), v.permute(0, 2, 1, 3)).view(B, Hkv, n, G, d)
    back = lambda t: t.transpose(1, 2).reshape(B, n, H, *t.shape[4:])  # noqa: E731
    return back(m), back(p.sum(-1)), back(acc)


def _finish(m, l, acc):
    some = l > 0
    o = torch.where(some.unsqueeze(-1), acc / l.unsqueeze(-1), torch.zeros_like(acc))
    lse = torch.where(some, m + torch.log(l), torch.full_like(m, -math.inf))
    return o.to(torch.bfloat16), lse.t().contiguous()


def _seen(nq, nk, most_q, most_k, causal):
    """[B, most_q, most_k]: key j of a sequence is seen by its query i (bottom-right aligned)."""
    i = torch.arange(most_q, device=DEV).view(1, -1, 1)
    j = torch.arange(most_k, device=DEV).view(1, 1, -1)
    nq, nk = nq.view(-1, 1, 1), nk.view(-1, 1, 1)
    seen = (j < nk) & (i < nq)
    return seen & (j <= i + nk - nq) if causal else seen


def _plain_decode(s):
    kc, vc, ke, ve = s["cache"]
    q, nq = _padded(s["q"].float(), s["cu_q"], s["max_q"])
    j = torch.arange(s["max_k"], device=DEV)
    page, off = s["table"].long()[:, j // s["page"]], j % s["page"]
    k = _values(kc.view(torch.uint8)[page, :, off].view(torch.float8_e4m3fn), ke[page, :, off])
    v = _values(vc.view(torch.uint8)[page, :, off].view(torch.float8_e4m3fn), ve[page, :, off])
    seen = _seen(nq, s["seqlens"].long(), q.shape[1], s["max_k"], s["causal"])
    parts = _softmax_parts(q, k, v, seen, s["scale"])
    b, i = _owners(s["cu_q"], s["q"].shape[0])
    return _finish(*(t[b, i] for t in parts))


def _plain_shared(s):
    n = s["q"].shape[0]
    q = s["q"].float()
    # the prefix: the queries of a group are the rows of one product
    cu_gq = s["cu_q"][s["cu_g"].long()]
    qg, ng = _padded(q, cu_gq, s["max_group"])
    kp, lp = _padded(s["kp"].float(), s["cu_p"], s["max_p"])
    vp, _ = _padded(s["vp"].float(), s["cu_p"], s["max_p"])
    seen = _seen(ng, lp, qg.shape[1], s["max_p"], False)
    g, i = _owners(cu_gq, n)
    m1, l1, a1 = (t[g, i] for t in _softmax_parts(qg, kp, vp, seen, s["scale"]))
    # the sequences' own keys
    qs, nq = _padded(q, s["cu_q"], s["max_q"])
    k, nk = _padded(s["k"].float(), s["cu_k"], s["max_k"])
    v, _ = _padded(s["v"].float(), s["cu_k"], s["max_k"])
    seen = _seen(nq, nk, qs.shape[1], s["max_k"], s["causal"])
    b, i = _owners(s["cu_q"], n)
    m2, l2, a2 = (t[b, i] for t in _softmax_parts(qs, k, v, seen, s["scale"]))
    m = torch.maximum(m1, m2)
    z = m.masked_fill(m == -math.inf, 0.0)
    w1, w2 = torch.exp(m1 - z), torch.exp(m2 - z)
    return _finish(m, l1 * w1 + l2 * w2, a1 * w1.unsqueeze(-1) + a2 * w2.unsqueeze(-1))


_PLAIN = dict(rope=_plain_rope, append=_plain_append, read=_plain_read, decode=_plain_decode,
              shared=_plain_shared)


# ------------------------------------------------------------------------------------- exact

def _code_values():
    """The values of the 256 e4m3 codes, from the format: sign, 4 bits of exponent biased by 7,
    3 bits of fraction; 0x7f and 0xff are NaN."""
    out = []
    for code in range(256):
        e, f = (code >> 3) & 15, code & 7
        v = f / 8 * 2.0 ** -6 if e == 0 else (1 + f / 8) * 2.0 ** (e - 7)
        v = math.nan if code & 127 == 127 else v
        out.append(-v if code & 128 else v)
    return torch.tensor(out, dtype=torch.float64, device=DEV)


def exact(c, seed):
    s = prepare(c, seed)
    f64 = torch.float64
    if c["op"] == "rope":
        n = sum(s["sections"])
        starts = [sum(s["sections"][:a]) for a in range(len(s["sections"]))]
        out = []
        for name in ("q", "k"):
            x = s[name].to(f64)
            y = x.clone()
            for a, size in enumerate(s["sections"]):
                for i in range(size):
                    p = starts[a] + i
                    inv = s["base"] ** -(i / size if s["per_axis"] else p / n)
                    u, w = (2 * p, 2 * p + 1) if s["interleaved"] else (p, p + n)
                    z = torch.polar(torch.ones(c["tokens"], 1, dtype=f64, device=DEV),
                                    s["pos"][a].to(f64).unsqueeze(1) * inv)
                    z = torch.complex(x[..., u], x[..., w]) * (z.conj() if c["inverse"] else z)
                    y[..., u], y[..., w] = z.real, z.imag
            out.append(y)
        return tuple(out)
    L = _lengths(c)
    if c["op"] in ("append", "read"):
        table = s["table"].cpu()
        val = _code_values()
        page = c["page"]
        if c["op"] == "append":
            # nearest code by distance, ties to the even one (the even last bit)
            pos = val[:127]
            mid = (pos[1:] + pos[:-1]) / 2
            kc, vc = (t.to(f64) for t in s["cache"][:2])
            for x, to in ((s["k"], kc), (s["v"], vc)):
                at = 0
                for b, n in enumerate(L["new"]):
                    y = x[at:at + n].to(f64)
                    at += n
                    if not n:
                        continue
                    size = y.abs().amax(-1, keepdim=True)
                    m, e = torch.frexp(size / 448)  # the least power of two over it: 2^e, or
                    e = torch.where(m > 0.5, e, e - 1).to(f64).clamp(-110, 120)  # itself
                    e = torch.where(size > 0, e, torch.zeros_like(e))
                    z = y * torch.exp2(-e)
                    lo = torch.searchsorted(mid, z.abs(), right=False)
                    hi = torch.searchsorted(mid, z.abs(), right=True)
                    i = torch.where(lo % 2 == 0, lo, hi)
                    z = torch.copysign(pos[i], z)
                    j = torch.arange(L["keys"][b] - n, L["keys"][b])
                    to[table[b, j // page].long().to(DEV), :, (j % page).to(DEV)] = z
            return kc, vc, None, None
        out = []
        for codes, exps in ((s["cache"][0], s["cache"][2]), (s["cache"][1], s["cache"][3])):
            rows = []
            for b, n in enumerate(L["keys"]):
                p = table[b, :-(-n // page)].long().to(DEV)
                x = (val[codes.view(torch.uint8)[p].long()]
                     * torch.exp2(exps[p].to(f64) - 127).unsqueeze(-1))
                rows.append(x.transpose(1, 2).reshape(-1, c["Hkv"], c["d"])[:n])
            out.append(torch.cat(rows))
        return tuple(out)
    # attention, sequence by sequence and head by head
    G = c["H"] // c["Hkv"]
    tokens = sum(L["new"])
    o = torch.zeros(tokens, c["H"], c["d"], dtype=f64, device=DEV)
    lse = torch.full((c["H"], tokens), -math.inf, dtype=f64, device=DEV)
    val, table, at, ak = _code_values(), s["table"].cpu() if "table" in s else None, 0, 0
    ap = [sum(L.get("prefix", ())[:g]) for g in range(c.get("groups", 0) + 1)]
    for b, (n, nk) in enumerate(zip(L["new"], L["keys"])):
        if c["op"] == "decode":
            p = table[b, :-(-nk // c["page"])].long().to(DEV)
            kv = [(val[s["cache"][t].view(torch.uint8)[p].long()]
                   * torch.exp2(s["cache"][t + 2][p].to(f64) - 127).unsqueeze(-1)
                   ).transpose(1, 2).reshape(-1, c["Hkv"], c["d"])[:nk] for t in (0, 1)]
            first = 0
        else:
            g = next(g for g in range(c["groups"]) if b < L["group"][g + 1])
            first = L["prefix"][g]
            kv = [torch.cat((s[pre][ap[g]:ap[g] + first], s[own_][ak:ak + nk])).to(f64)
                  for pre, own_ in (("kp", "k"), ("vp", "v"))]
        ak += nk
        for i in range(n):
            most = first + (max(0, min(nk, i + nk - n + 1)) if c["causal"] else nk)
            if most:
                k, v = (x[:most].transpose(0, 1) for x in kv)  # [Hkv, keys, d]
                q = s["q"][at + i].to(f64).view(c["Hkv"], G, c["d"])
                x = torch.matmul(q, k.transpose(1, 2)) * s["scale"]
                w = torch.logsumexp(x, -1)
                lse[:, at + i] = w.reshape(-1)
                o[at + i] = torch.matmul(torch.exp(x - w.unsqueeze(-1)), v).reshape(c["H"], -1)
        at += n
    return o, lse
