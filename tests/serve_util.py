"""Plain 64-bit references of the serving operators (rotary positions, the e4m3 cache, attention
over it), in numpy, and the rounding bounds the tests hold the kernels to."""
from __future__ import annotations

import math
from decimal import Decimal, getcontext

import numpy as np
import torch

getcontext().prec = 60
TWO_PI = Decimal("6.28318530717958647692528676655900576839433879875021164194988918")

# half a step of a type, relative to the value
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def code_values() -> np.ndarray:
    """The 256 e4m3 codes' values (1 sign, 4 exponent bits biased by 7, 3 fraction bits; 0x7f
    and 0xff are NaN)."""
    c = np.arange(256)
    e, f = (c >> 3) & 15, (c & 7) / 8.0
    v = np.where(e == 0, f * 2.0 ** -6, (1 + f) * 2.0 ** (e - 7.0))
    v[(c & 127) == 127] = np.nan
    return np.where(c & 128, -v, v)


CODES = code_values()


def quantise_row(x: np.ndarray):
    """(codes, exponent byte) of one row by the definition: the least power of two with max|x| <=
    448 * 2^e, e in [-110, 120], values to the nearest code, ties to the even one."""
    finite = np.isfinite(x)
    size = np.abs(x[finite]).max() if finite.any() else 0.0
    e = 0
    if size > 0:
        e = math.frexp(size / 448.0)[1] - (math.frexp(size / 448.0)[0] == 0.5)
        e = min(max(e, -110), 120)
    pos = CODES[:127]
    out = np.zeros(x.shape, np.uint8)
    for i, v in enumerate(x):
        if not np.isfinite(v):
            out[i] = 0x7F
            continue
        y = abs(float(v)) * 2.0 ** -e
        near = np.abs(pos - y)
        best = np.flatnonzero(near == near.min())
        c = best[0] if len(best) == 1 or best[0] % 2 == 0 else best[1]
        out[i] = c | (0x80 if math.copysign(1.0, v) < 0 else 0)
    return out, e + 127


def values(codes: np.ndarray, exps: np.ndarray) -> np.ndarray:
    """fp64 values of codes [..., d] under exponent bytes [...]."""
    return CODES[codes] * np.exp2(exps.astype(np.float64) - 127.0)[..., None]


def attention_rows(q, k, v, scale, causal, shift, v_scale=None, always=0):
    """One (sequence, head): q [nq, d], k, v [nk, d] fp64.  Query i sees key j iff j <= i + shift
    (every key without the mask), and the first `always` keys whatever the mask.  Returns o, lse, and for the error bound sum_j p_j |v_j|, the
    largest scale * sum |q| |k| of each row and (v_scale: the power of two of each V row) the
    floor 2^-36 * max_j (p_j 2^ev_j) * sum_j |v_j| / 2^ev_j, else 0.  A row that sees no key: o = 0,
    lse = -inf."""
    nq, d = q.shape
    nk = k.shape[0]
    o, pv = np.zeros((nq, d)), np.zeros((nq, d))
    lse, mag, low = np.full(nq, -np.inf), np.zeros(nq), np.zeros((nq, d))
    for i in range(nq):
        n = nk if not causal else max(always, min(nk, i + shift + 1))
        if n == 0:
            continue
        with np.errstate(invalid="ignore", over="ignore"):
            x = (k[:n] @ q[i]) * scale
            mag[i] = np.abs(scale) * np.nanmax(np.abs(k[:n]) @ np.abs(q[i]))
            m = x.max()
            p = np.exp(x - m)
            lse[i] = m + np.log(p.sum())
            p /= p.sum()
            o[i] = p @ v[:n]
            pv[i] = p @ np.abs(v[:n])
            if v_scale is not None:
                s = v_scale[:n]
                low[i] = 2.0 ** -36 * (p * s).max() * (np.abs(v[:n]) / s[:, None]).sum(0)
    return o, lse, pv, mag, low


def check_rows(o, lse, ref_o, ref_lse, pv, mag, low, weight_step, what=""):
    """o [.., d] bf16 and lse fp32 against the reference.  Bounds, from the arithmetic:
      - a logit's fp32 accumulation over d terms in k-steps of 16, each good to 2^-23 of the
        magnitudes summed: dx <= 2^-19 * scale * sum |q||k| (and 2^-22 for its base-2 copy);
      - the weights are rounded to `weight_step` (relative) and exp2 is good to 2^-22: with a
        logit error dx each weight moves by 2 dx (its own and the sum's), so
        |dO| <= (weight_step + 2 dx + 2^-18) * sum p|v|;
      - f16 weights multiply V's codes in a frame where the largest weight (with its row's scale)
        is at least 2^11 and f16's smallest step is 2^-24: each key's weight is off by at most
        2^-25, i.e. 2^-36 of the largest, times its code: `low`;
      - O is rounded to bf16: 2^-8 |O|; lse: dx + 2^-20 (1 + |lse|)."""
    o, lse = o.double().cpu().numpy(), lse.double().cpu().numpy()
    bad = np.isnan(ref_o) | (np.abs(ref_o) > 3.0e38)
    assert (np.isnan(o) == np.isnan(ref_o)).all() or bad.any(), f"NaN pattern {what}"
    assert (np.isnan(o)[~bad] == False).all(), f"NaN in O {what}"  # noqa: E712
    assert np.isnan(o[np.isnan(ref_o)]).all(), f"missing NaN {what}"
    assert ((lse == -np.inf) == (ref_lse == -np.inf)).all(), f"empty rows {what}"
    dx = 2.0 ** -19 * mag + 2.0 ** -22 * (1 + np.abs(np.where(np.isfinite(ref_lse), ref_lse, 0)))
    tol = 2.0 ** -8 * np.abs(ref_o) + (weight_step + 2 * dx + 2.0 ** -18)[..., None] * pv + low + 1e-38
    err = np.abs(o - ref_o)
    over = (err > tol) & ~bad
    assert not over.any(), (what, float((err / tol)[~bad].max()), np.argwhere(over)[:5].tolist())
    some = np.isfinite(ref_lse)
    lerr = np.abs(lse[some] - ref_lse[some])
    ltol = (dx + 2.0 ** -20 * (1 + np.abs(ref_lse)))[some]
    assert (lerr <= ltol).all(), (what, float((lerr / ltol).max()))
    return float((err / tol)[~bad].max()) if (~bad).any() else 0.0


def rope_reference(x, pos, inv_freq, axis, interleaved, inverse):
    """x [total, heads, d] fp64, pos [axes, total] ints: angles reduced in 60 decimal digits."""
    n = len(inv_freq)
    y = x.copy()
    for p in range(n):
        f = Decimal(inv_freq[p])
        ang = [float((Decimal(int(t)) * f) % TWO_PI) for t in pos[axis[p]]]
        c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]
        if inverse:
            s = -s
        i, j = (2 * p, 2 * p + 1) if interleaved else (p, n + p)
        y[..., i] = x[..., i] * c - x[..., j] * s
        y[..., j] = x[..., j] * c + x[..., i] * s
    return y
