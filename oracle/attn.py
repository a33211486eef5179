"""Plain fp64 reference of the attention operators (numpy, loops over sequences, heads and tokens).
Test infrastructure only: the product path never loads it."""
from __future__ import annotations

import math

import numpy as np


def rope(x, positions, freq, interleaved, mscale):
    """x [T, H, D]: pair i of each head turned by the angle positions[t] * freq[i], times mscale.  The
    angle is taken in extended precision (64-bit significand): a position of 2^40 times a frequency of
    1 leaves 2^-24 of a radian there, and only 2^-13 in fp64."""
    x = np.array(x, np.float64)
    h = len(freq)
    angle = np.asarray(positions, np.longdouble)[:, None] * np.asarray(freq, np.longdouble)[None, :]
    cos, sin = (f(angle).astype(np.float64)[:, None, :] * mscale for f in (np.cos, np.sin))
    ia = np.arange(h) * 2 if interleaved else np.arange(h)
    ib = ia + 1 if interleaved else ia + h
    a, b = x[..., ia].copy(), x[..., ib].copy()
    x[..., ia], x[..., ib] = a * cos - b * sin, b * cos + a * sin
    return x


E4M3 = np.array(sorted({(m / 8 if e == 0 else 1 + m / 8) * 2.0 ** (max(e, 1) - 7)
                        for e in range(16) for m in range(8) if not (e == 15 and m == 7)}))


def to_e4m3(x):
    """Nearest e4m3 value, ties to the even code, saturated at 448 (the codes of E4M3 are in order, so
    an even place is an even mantissa)."""
    mag = np.minimum(np.abs(np.asarray(x, np.float64)), 448.0)
    hi = np.clip(np.searchsorted(E4M3, mag), 1, len(E4M3) - 1)
    lo = hi - 1
    dl, dh = mag - E4M3[lo], E4M3[hi] - mag
    pick = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    return np.copysign(E4M3[pick], x)


def quantize(x, kind):
    """Rows x [..., D] (fp32 values) -> (code values, scales): the fp32 operations of the definition."""
    x = np.asarray(x, np.float32)
    top = np.float32(127.0 if kind == "int8" else 448.0)
    amax = np.abs(x).max(-1)
    live = amax >= np.float32(2.0 ** -100)
    safe = np.where(live, amax, np.float32(1))
    scale = np.where(live, safe * (np.float32(1) / top), np.float32(0))
    mult = np.where(live, (np.float32(1) / safe) * top, np.float32(0))
    y = np.clip(x * mult[..., None], -top, top)
    return (np.rint(y).astype(np.float64) if kind == "int8" else to_e4m3(y)), scale


def attend(q, k, v, scale, seen):
    """q [H, D] rows of one query token's heads that share k, v [n, D]; the first `seen` keys count.
    Returns (out [H, D], lse [H], sum of |weight * v| [H, D], largest |scaled score| [H], largest
    scaled sum of |q k| [H])."""
    q, k, v = (np.asarray(t, np.float64) for t in (q, k[:seen], v[:seen]))
    H, D = q.shape
    if seen <= 0:
        z = np.zeros((H, D))
        return z, np.full(H, -math.inf), z, np.zeros(H), np.zeros(H)
    s = scale * (q @ k.T)
    m = s.max(-1, keepdims=True)
    p = np.exp(s - m)
    l = p.sum(-1, keepdims=True)
    return ((p / l) @ v, (m + np.log(l))[:, 0], (p / l) @ np.abs(v), np.abs(s).max(-1),
            scale * (np.abs(q) @ np.abs(k).T).max(-1))


def _stack(results, T, Hq, D):
    out = [np.zeros((T, Hq, D)), np.full((T, Hq), -math.inf), np.zeros((T, Hq, D)), np.zeros((T, Hq)),
           np.zeros((T, Hq))]
    for t, h, r in results:
        for o, x in zip(out, r):
            o[t, h] = x
    return out


def prefill(q, k, v, cu_q, cu_k, causal, scale):
    """attend() for every token of every packed sequence; rows of no sequence stay zero."""
    T, Hq, D = q.shape
    G = Hq // k.shape[1]
    res = []
    for b in range(len(cu_q) - 1):
        lq, lk = cu_q[b + 1] - cu_q[b], cu_k[b + 1] - cu_k[b]
        for i in range(lq):
            seen = max(0, min(lk, i + 1 + lk - lq)) if causal else lk
            for h in range(k.shape[1]):
                hs = slice(h * G, (h + 1) * G)
                rows = slice(cu_k[b], cu_k[b + 1])
                res.append((cu_q[b] + i, hs, attend(q[cu_q[b] + i, hs], k[rows, h], v[rows, h], scale, seen)))
    return _stack(res, T, Hq, D)


def decode(q, k, v, table, lens, scale):
    """k, v [pages, Hkv, page, D] as values.  Tokens on pages outside the cache are not seen."""
    B, Hq, D = q.shape
    pages, Hkv, page, _ = k.shape
    G = Hq // Hkv
    res = []
    for b in range(B):
        n = max(0, min(int(lens[b]), table.shape[1] * page))
        at = [(int(table[b, j // page]), j % page) for j in range(n) if 0 <= table[b, j // page] < pages]
        for h in range(Hkv):
            kk = np.array([k[p, h, o] for p, o in at]).reshape(len(at), D)
            vv = np.array([v[p, h, o] for p, o in at]).reshape(len(at), D)
            hs = slice(h * G, (h + 1) * G)
            res.append((b, hs, attend(q[b, hs], kk, vv, scale, len(at))))
    return _stack(res, B, Hq, D)


def attention_tolerance(io_half, weight_half, out, mag, smax, qkmax, D, keys):
    """How far an attention output may be off.  Scores are sums of D fp32 products (at most D + 4
    roundings of 2^-24 of the summed magnitudes), scaled and shifted in fp32 (2^-22 of the score), so a weight is off by twice
    that relative to the maximum, the sum by as much again; the exponential adds 2^-22, the sums over
    the keys 2^-24 each, the rounding of a weight weight_half; all of it relative to sum |w v|.  The result is rounded
    once to the io dtype."""
    eps = (D + 4) * 2.0 ** -24 * qkmax + 2.0 ** -22 * smax
    rel = weight_half + 4 * eps + 2.0 ** -20 + 2 * keys * 2.0 ** -24
    return io_half * np.abs(out) + rel[..., None] * mag, 2 * eps + keys * 2.0 ** -24 + 2.0 ** -20
