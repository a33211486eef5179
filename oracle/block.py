"""Plain fp64 reference of the residual norm and of 4-bit weights (numpy).  Test infrastructure only: the product path never
loads it."""
from __future__ import annotations

import numpy as np

from .attn import to_e4m3

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
TINY = 2.0 ** -100


def rms_norm(h, weight, eps):
    """h [T, D]: each row over its root mean square, times weight."""
    h = np.asarray(h, np.float64)
    return h / np.sqrt((h * h).mean(-1, keepdims=True) + eps) * np.asarray(weight, np.float64)


def row_codes(y):
    """(code values, scales) of rows in e4m3, without the roundings of the scale."""
    y = np.asarray(y, np.float64)
    amax = np.abs(y).max(-1)
    live = amax >= TINY
    safe = np.where(live, amax, 1.0)
    return np.where(live[:, None], to_e4m3(y * (448.0 / safe)[:, None]), 0.0), np.where(live, amax / 448.0, 0.0)


def quantize(w):
    """w [M, K] -> (codes 0 .. 15 [M, K], scale bytes [M, ceil(K / 32)]), value by value from the definition."""
    w = np.asarray(w, np.float64)
    M, K = w.shape
    codes, scales = np.zeros((M, K), np.uint8), np.zeros((M, -(-K // 32)), np.uint8)
    for m in range(M):
        for g in range(scales.shape[1]):
            x = w[m, 32 * g:32 * g + 32]
            amax = np.abs(x).max()
            if amax < TINY:
                scales[m, g] = 127
                continue
            f, n = np.frexp(amax)  # amax = f 2^n, f in [0.5, 1): three significant bits of f are eighths
            n = int(n) - 1 + (1 if f >= 7 / 8 else 0)
            e = min(n - 2 + 127, 252)
            scales[m, g] = e
            for i, v in enumerate(np.abs(x) * 2.0 ** (127 - e)):
                d = np.abs(E2M1 - min(v, 6.0))
                near = np.flatnonzero(d == d.min())  # one, or two neighbours: the even code of them
                c = near[0] if len(near) == 1 or near[0] % 2 == 0 else near[1]
                codes[m, 32 * g + i] = c + (8 if np.signbit(x[i]) else 0)
    return codes, scales


def dequantize(codes, scales):
    """The weight that rows of codes and scale bytes stand for."""
    c = np.asarray(codes).astype(int)
    mag = E2M1[c % 8] * np.where(c >= 8, -1.0, 1.0)
    s = np.repeat(np.asarray(scales).astype(np.float64), 32, axis=1)[:, :c.shape[1]]
    return mag * 2.0 ** (s - 127)


def unpack(codes, scales, M, K):
    """Rows of codes and scale bytes from the packed layout, byte by byte."""
    codes, scales = np.asarray(codes), np.asarray(scales)
    c, s = np.zeros((M, K), np.uint8), np.zeros((M, -(-K // 32)), np.uint8)
    for m in range(M):
        for k in range(K):
            byte = codes[m // 16, k // 128, (k % 128) // 32 * 16 + m % 16, (k % 32) // 2]
            c[m, k] = byte % 16 if k % 2 == 0 else byte // 16
            if k % 32 == 0:
                s[m, k // 32] = scales[m // 16, k // 512, (k % 128) // 32 * 16 + m % 16, (k // 128) % 4]
    return c, s
