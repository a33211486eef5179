"""Values beside the border between two codes: what a row's 8-bit codes need fp64 products for.  The same rows in the arithmetic of
fp32, rounded at each step, come out with other codes (no GPU): so test_gpu_block_codes.py tells the two apart."""
import numpy as np
import pytest

from oracle import attn as A

CODES = np.unique(np.abs(A.to_e4m3(np.linspace(0, 448, 1 << 16))))  # every magnitude


def beside_borders(T, D, seed=0):
    """(rows [T, D] fp32, their codes): values next to where a code begins, more than half a step of fp32 away, so that rounding
    the exact product to fp32 once changes none, and at most 3 * 2^-24 of their size."""
    rng = np.random.default_rng(seed)
    top = (1 + rng.random((T, 1))).astype(np.float32)
    low = rng.integers(40, len(CODES) - 1, (T, D))  # codes from 2^-3 or so on
    border = (CODES[low] + CODES[low + 1]) / 2
    v = (border * top.astype(np.float64) / 448).astype(np.float32)
    way = rng.integers(-2, 3, (T, D))
    for step in (1, 2):
        v = np.where(np.abs(way) >= step, np.nextafter(v, np.where(way > 0, np.float32(9), np.float32(0))), v)
    # exact: 448 has 3 significant bits, a border 5, the others 24
    left, right = v.astype(np.float64) * 448, border * top.astype(np.float64)
    off = np.abs(left - right) / right
    keep = (off > 1.01 * np.spacing(border.astype(np.float32)).astype(np.float64) / 2 / border) & (off < 3 * 2.0 ** -24)
    codes = np.where(left > right, CODES[low + 1], CODES[low])
    v, codes = np.where(keep, v, 0), np.where(keep, codes, 0)
    sign = np.where(rng.integers(0, 2, (T, D)) == 1, np.float32(-1), np.float32(1))
    place = rng.integers(0, D, T)
    x, c = v * sign, codes * sign
    x[np.arange(T), place], c[np.arange(T), place] = top[:, 0], 448
    assert keep.mean() > 0.3
    return x.astype(np.float32), c


def test_the_rows_codes_are_the_definition_s():
    x, c = beside_borders(20, 256)
    top = np.abs(x).max(-1, keepdims=True).astype(np.longdouble)
    y = np.abs(x.astype(np.longdouble)) * 448 / top  # 64 bits: the borders are 2^-24 away
    want = CODES[np.abs(y[..., None] - CODES).argmin(-1)] * np.sign(x)
    assert np.array_equal(want, c)


@pytest.mark.parametrize("D", [64, 4096])
def test_fp32_products_give_other_codes(D):
    x, c = beside_borders(4096 // D * 32, D)
    f, ss = np.float32, (x.astype(np.float64) ** 2).mean(-1, keepdims=True)
    r = f(1) / np.sqrt(ss.astype(f))
    for scaled in (r, np.exp2(np.floor(np.log2(r))).astype(f)):  # y over its largest, and h over its largest
        y = x * scaled
        got = A.to_e4m3((y * (f(448) / np.abs(y).max(-1, keepdims=True))).astype(f))
        assert (got != c).sum() > 20
    got = A.to_e4m3((x.astype(np.float64) * (448 / np.abs(x).max(-1, keepdims=True).astype(np.float64))).astype(f))
    assert np.array_equal(got, c)  # fp64, rounded to fp32 before
