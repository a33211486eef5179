"""The precision bound of tests/attn_precision.py: attention emulated in the kernels' number formats is within it, and with a
part left out, a step of keys dropped or a row of values misplaced it is not."""
import numpy as np
import pytest

from tests import attn_precision as P

F = np.float32


def product(a, b, n):
    """a @ b of fp32 by n bf16 parts of each, the products of which the first n orders are kept, the small ones first."""
    a, b = P.parts(a, n), P.parts(b, n)
    s = F(0)
    for order in reversed(range(n)):
        for i in range(order + 1):
            s = s + a[i] @ b[order - i]
    return s


def emulated(q, k, v, scale, qk, pv, drop=None, misplace=None):
    """One head in fp32: q [R, D] against all of k, v [n, D]; qk and pv are the two products."""
    s = qk(q, k.T) * F(scale * np.log2(np.e))
    if drop is not None:
        s[:, drop] = -np.inf
    m = s.max(-1, keepdims=True)
    p = np.exp2(s - m)
    total = p.sum(-1, keepdims=True)
    if misplace is not None:
        v = v.copy()
        v[misplace] = v[misplace][::-1]
    return pv(p, v) / total, (m + np.log2(total))[:, 0] * F(np.log(2))


def inputs(seed, R, n, D, io):
    rng = np.random.default_rng(seed)
    k, v = P.keys_values(rng, n, (D,), io)
    q = rng.standard_normal((R, D))
    return [(P.bf16 if io == "bf16" else F)(x) for x in (q, k, v)]


def judged(seed, R, n, D, io, c, qk, pv, **kw):
    q, k, v = inputs(seed, R, n, D, io)
    scale = D ** -0.5
    ref = P.definition(*(x.astype(np.float64) for x in (q, k, v)), np.full(R, n), scale)
    out, lse = emulated(q, k, v, scale, qk, pv, **kw)
    return P.excess(P.bf16(out) if io == "bf16" else out, ref, P.HALF[io], c, lse)


plain = lambda a, b: a @ b  # noqa: E731
SIZES = [(40, 300, 64), (12, 1000, 128), (8, 2000, 256), (6, 20011, 72)]


@pytest.mark.parametrize("R,n,D", SIZES)
def test_fp32_prompts(R, n, D):
    three, two = (lambda a, b: product(a, b, 3)), (lambda a, b: product(a, b, 2))
    assert judged(1, R, n, D, "f32", P.C_F32, three, three)[1] < 0.7
    assert judged(1, R, n, D, "f32", P.C_F32, two, three)[1] > 1.5   # q and k without their third parts
    cut = lambda x: np.sum(P.parts(x, 2), 0, dtype=F)  # noqa: E731
    for one in (lambda a, b: product(cut(a), b, 3), lambda a, b: product(a, cut(b), 3)):  # one operand of the two
        assert judged(1, R, n, D, "f32", P.C_F32, one, three)[1] > 1.5
        assert judged(1, R, n, D, "f32", P.C_F32, three, one)[1] > 1.5
    assert judged(1, R, n, D, "f32", P.C_F32, three, two)[1] > 1.5   # weights and values


@pytest.mark.parametrize("R,n,D", SIZES)
def test_fp32_decode_on_codes(R, n, D):
    """Codes are exact in bf16; q and the weights times the rows' scales are split."""
    def split(parts_of_a):
        return lambda a, b: sum((x @ b for x in reversed(P.parts(a, parts_of_a))), F(0))

    def run(nq, nw):
        rng = np.random.default_rng(2)
        k, v = P.keys_values(rng, n, (D,), "f32")
        ks, vs = (np.abs(x).max(-1, keepdims=True) / 127 for x in (k, v))
        kc, vc = np.rint(k / ks).astype(F), np.rint(v / vs).astype(F)
        ks, vs, q, scale = ks.astype(F), vs.astype(F), rng.standard_normal((R, D)).astype(F), D ** -0.5
        ref = P.definition(q.astype(np.float64), kc * ks.astype(np.float64), vc * vs.astype(np.float64), np.full(R, n), scale)
        got, lse = emulated(q, kc, vc, scale, lambda a, b: split(nq)(a, b) * ks[:, 0], lambda p, x: split(nw)(p * vs[:, 0], x))
        return P.excess(got, ref, P.HALF["f32"], P.C_F32, lse)[1]
    assert run(3, 3) < 0.7 and run(2, 3) > 1.5 and run(3, 2) > 1.5


@pytest.mark.parametrize("R,n,D", SIZES)
def test_bf16_decode(R, n, D):
    def weights(parts):
        return lambda p, v: sum((x @ v for x in reversed(P.parts(p, parts))), F(0))
    assert judged(3, R, n, D, "bf16", P.C_DECODE, plain, weights(2))[1] < 0.7
    assert judged(3, R, n, D, "bf16", P.C_DECODE, plain, weights(1))[1] > 1.5   # without their second part
    assert judged(3, R, n, D, "bf16", P.C_PROMPT, plain, weights(1))[1] < 0.7   # as prompts have them


@pytest.mark.parametrize("io,c", [("f32", P.C_F32), ("bf16", P.C_DECODE), ("bf16", P.C_PROMPT)])
@pytest.mark.parametrize("n", [300, 2500, 20011])
def test_dropped_and_misplaced_keys(io, c, n):
    """A step of 32 keys not counted, the values of 256 keys in reverse order, of 4 keys; values of random sign, whose output
    is as large as its noise."""
    for kw in (dict(drop=slice(64, 96)), dict(misplace=slice(32, 288)), dict(misplace=slice(100, 104))):
        rng = np.random.default_rng(4)
        q, k, v = ((P.bf16 if io == "bf16" else F)(rng.standard_normal(s)) for s in ((8, 64), (n, 64), (n, 64)))
        ref = P.definition(*(x.astype(np.float64) for x in (q, k, v)), np.full(8, n), 0.125)
        for broken in (False, True):
            out, lse = emulated(q, k, v, 0.125, plain, plain, **(kw if broken else {}))
            got = P.excess(P.bf16(out) if io == "bf16" else out, ref, P.HALF[io], c, lse)
            assert got[1] > 1.2 if broken else got[1] < 0.7, (kw, got)


def test_three_parts_hold_what_fp32_holds_up_to_two_to_127():
    """Nothing is left of 24 bits, up to 2^127; from half a step of bf16 below 2^128 on, a value rounds to infinity."""
    rng = np.random.default_rng(5)
    x = rng.uniform(-2, 2, 10000).astype(F)
    for e in (0, 60, 126):
        y = x * F(2.0 ** e)
        h, m, l = P.parts(y, 3)
        assert np.array_equal((h.astype(np.float64) + m + l).astype(F), y)
        assert np.all(np.abs(y.astype(np.float64) - h - m - l) <= 2.0 ** -26 * np.abs(y))
    with np.errstate(over="ignore", invalid="ignore"):
        assert np.isinf(P.bf16(F([3.4e38]))).all() and np.isfinite(P.bf16(F([2.0 ** 127]))).all()
