"""How precise the attention operators are, as a whole: a bound on the root mean square of the error, which a lost part of
an operand, a dropped step of keys or a row in the wrong place exceeds by far, where bounds on single values that add up
every rounding at its worst let them pass.  Shared by the CPU tests of the bound and the GPU tests of the kernels.

Weights w_j (their sum 1) of values v_j that are independent in sign: errors of the weights that are independent of
one another, each eps of its weight, leave eps * noise in the output, noise = sqrt(sum_j (w_j v_j)^2).  The bound is
  rms(error) <= half * rms(out) + c * rms(noise)
over all outputs, and four times that over the channels of any one row.  half: half a step of the io dtype, the output's
own rounding (bf16 2^-8, fp32 2^-24).  c:
  fp32, 2^-20.  A rounding to fp32 is off by 0.4 * 2^-24 (rms over all mantissas).  A score is a sum of at most 6 * 256 / 16 = 96
    products of the matrix cores, whose partial sums are 0.6 of it (rms): sqrt(96) * 0.6 * 0.4 = 2.4 roundings, of
    scores of size 1; scaling and shifting a score of up to 5 adds 2 * 5 * 0.4 = 4; the exponential 2.  An output is a sum over at most
    1000 keys of a wave, 16 at a time and six times: sqrt(375) * 0.6 * 0.4 = 4.7.  Together, as they are independent, 7 * 2^-24;
    what three bf16 parts leave out is below one.  16 * 2^-24 is twice that.
  bf16 decode, 2^-16.  A weight is the sum of two bf16, 2^-17 at most; twice that for the terms above.
  bf16 prompts, 2^-8.  A weight is rounded to bf16 once, 2^-8 at most.
lse: scores as above, 7 * 2^-24 (rms) of a few; the largest of 10^5 rows is 4.5 times the rms: 2^-19, and 2^-22 of lse for
its logarithm and last product."""
import numpy as np

HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
C_F32, C_DECODE, C_PROMPT = 2.0 ** -20, 2.0 ** -16, 2.0 ** -8


def bf16(x):
    """fp32 values rounded to bf16 (nearest even)."""
    u = np.ascontiguousarray(x, np.float32).view(np.uint32).astype(np.uint64)
    u = u + 0x7FFF + ((u >> 16) & 1)
    return (u & 0xFFFF0000).astype(np.uint32).view(np.float32)


def parts(x, n):
    """fp32 values as n bf16, each the remainder of the last, rounded."""
    res = []
    x = np.asarray(x, np.float32)
    for _ in range(n):
        res.append(bf16(x))
        x = x - res[-1]
    return res


def definition(q, k, v, seen, scale):
    """q [R, D], k, v [n, D], row i sees the first seen[i] keys, all fp64: (out, lse, noise) of one head."""
    s = np.where(np.arange(len(k))[None] < np.asarray(seen)[:, None], scale * (q @ k.T), -np.inf)
    some = np.asarray(seen) > 0
    m = np.where(some, s.max(-1, initial=-np.inf), 0.0)
    p = np.exp(s - m[:, None])
    total = np.where(some, p.sum(-1), 1.0)
    w = p / total[:, None]
    return w @ v, np.where(some, m + np.log(total), -np.inf), np.sqrt((w * w) @ (v * v))


def prompt(q, k, v, cu_q, cu_k, causal, scale, tokens=None):
    """definition() of every head of packed sequences [T, H, D], or of the given tokens (indices into q's rows)."""
    T, Hq, D = q.shape
    G = Hq // k.shape[1]
    out, lse, noise = np.zeros((T, Hq, D)), np.full((T, Hq), -np.inf), np.zeros((T, Hq, D))
    wanted = np.ones(T, bool) if tokens is None else np.isin(np.arange(T), tokens)
    for b in range(len(cu_q) - 1):
        lq, lk = cu_q[b + 1] - cu_q[b], cu_k[b + 1] - cu_k[b]
        rows = np.arange(cu_q[b], cu_q[b + 1])
        rows = rows[wanted[rows]]
        i = rows - cu_q[b]
        seen = np.clip(i + 1 + lk - lq, 0, lk) if causal else np.full(len(rows), lk)
        keys = slice(cu_k[b], cu_k[b + 1])
        for h in range(Hq):
            if len(rows):
                out[rows, h], lse[rows, h], noise[rows, h] = definition(q[rows, h], k[keys, h // G], v[keys, h // G], seen, scale)
    return (out, lse, noise) if tokens is None else tuple(x[wanted] for x in (out, lse, noise))


def rms(x, axis=None):
    return np.sqrt(np.mean(np.square(x), axis=axis))


def excess(got, ref, half, c, lse=None):
    """By what the outputs exceed the bounds, as (what, factor) of the worst: 1 or less is within."""
    out, rlse, noise = ref
    err = np.asarray(got, np.float64) - out
    if not np.all(np.isfinite(err)):
        return "not finite", np.inf
    if err.size == 0:
        return "nothing", 0.0
    bound = lambda axis: half * rms(out, axis) + c * rms(noise, axis)  # noqa: E731
    tiny = 2.0 ** -120  # rows of zeros are to be zero
    worst = [("rms", rms(err) / (bound(None) + tiny)), ("rms of a row", (rms(err, -1) / (4 * bound(-1) + tiny)).max())]
    if lse is not None:
        empty = np.isneginf(rlse)
        l = np.asarray(lse, np.float64)
        if not np.array_equal(np.isneginf(l), empty):
            return "lse of rows without keys", np.inf
        at = np.where(empty, 0, rlse)
        worst.append(("lse", (np.abs(np.where(empty, 0, l) - at) / (2.0 ** -19 + 2.0 ** -22 * np.abs(at))).max()))
    return max(worst, key=lambda x: x[1])


def keys_values(rng, n, shape, io, spread=0.05):
    """Keys and values [n, *shape].  For bf16 in pairs of nearly equal keys with opposite values: an output is what the weights
    of a pair differ by, far below its noise, so that its own rounding does not hide an error of the weights.  (For
    fp32 that rounding is small, and pairs would hide an error of q, which shifts both scores alike.)"""
    if io == "f32":
        return rng.standard_normal((n, *shape)), rng.standard_normal((n, *shape))
    half = -(-n // 2)
    k, v = rng.standard_normal((half, *shape)), rng.standard_normal((half, *shape))
    k2 = k + spread * rng.standard_normal(k.shape)
    order = rng.permutation(2 * half)[:n]
    return np.concatenate([k, k2])[order], np.concatenate([v, -v])[order]
