"""The residual norm and the 4-bit projections on the GPU against their fp64 definitions (oracle/block.py): sizes, types,
strides and values where they can go wrong.  Tolerances count roundings, u = 2^-24 for fp32 and half a step of an output's type
once at the end (relative: bf16 2^-8, fp32 2^-24, e4m3 2^-4).

Norm: a thread adds at most 32 squares, the wave and the workgroup up to 22 times more, so the mean of squares is within 56 u
with its division and eps; the root halves that, rsqrt is within 2 u, two products: 32 u = 2^-19 of a value.
Linear: products are exact and the sum of K of them, each addition within 2^-23 of its partial sum whatever its order, is
within K 2^-23 of the sum of magnitudes.  As a whole: partial sums of i terms of independent signs are about sqrt(i) of one,
so K additions leave 2^-23 sqrt(K / 2) of a result's size.
e4m3 tokens with a bf16 output: the instruction that takes codes drops from a product what is below 2^-13 of the largest of
its eight columns' (test_what_the_instruction_on_codes_keeps), at most 2^-13 of their magnitudes' sum for each of the eight:
2^-10 of the sum of magnitudes in all."""
import numpy as np
import pytest
import torch

import selective_state_space_causal_amd as ssm
from oracle import block as O
from selective_state_space_causal_amd import block as B

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
E4M3 = torch.float8_e4m3fn
DT = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": E4M3}
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
NORM = 2.0 ** -19


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def rnd(seed, *shape, scale=1.0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * scale


def framed(t, pad, fill):
    """t [T, D] as a view in the middle of a larger tensor of `fill`, and that tensor."""
    big = torch.full((t.shape[0] + 3, t.shape[1] + pad), fill, dtype=torch.float32).to(t.dtype).to(DEV)
    view = big[:t.shape[0], :t.shape[1]]
    view.copy_(t)
    return view, big


def close(got, want, tol, what):
    got = f64(got)
    assert got.shape == want.shape and np.all(np.isfinite(got)), f"{what}: shape or not finite"
    bad = np.abs(got - want) - tol
    assert bad.max() <= 0, f"{what}: {np.abs(got - want).max():.3e} off, {bad.max():.3e} over the bound"


# ---------------------------------------------------------------- the norm

def check_norm(T, D, io, res, q8, seed=0, eps=1e-5, x=None, pad=0, in_place=False):
    dt = DT[io]
    x = (rnd(seed, T, D) if x is None else x).to(dt)
    r = None if res is None else rnd(seed + 1, T, D, scale=3.0).to(DT[res])
    w = (1 + 0.3 * rnd(seed + 2, D)).to(DEV)
    xv, xbig = framed(x, pad, float("nan"))
    rv = rbig = None
    if r is not None:
        rv, rbig = framed(r, pad, float("nan"))
    out, obig = framed(torch.zeros(T, D).to(E4M3 if q8 else dt), pad, 7.0)
    if in_place and not q8:
        out, obig = xv, xbig
    ro = None if r is None or in_place else framed(torch.zeros(T, D).to(r.dtype), pad, 7.0)
    ret = ssm.rms_norm(xv, w, residual=rv, residual_out=None if ro is None else ro[0], eps=eps, out=out)
    y, s = ret if q8 else (ret, None)
    assert y is out
    h = x if r is None else (x.float() + r.float()).to(r.dtype)
    what = f"norm {T}x{D} {io} {res} {q8}"
    if r is not None:
        stored = rv if in_place else ro[0]
        assert torch.equal(stored.cpu(), h), f"{what}: residual"
        if not in_place:
            assert torch.equal(rv.cpu(), r), f"{what}: residual is an input"
    want = O.rms_norm(f64(h), f64(w), eps)
    if q8:
        amax = np.abs(want).max(-1)
        close(s, amax / 448, amax / 448 * 2.0 ** -18, what + " scale")
        val = f64(y) * f64(s)[:, None]
        step = f64(s)[:, None] * (np.abs(f64(y)) * 2.0 ** -4 + 2.0 ** -10)
        assert np.all(np.abs(val - want) <= step + np.abs(want) * 2.0 ** -18), what
        codes, _ = O.row_codes(want)
        # the whole: nearly all codes are those of the definition (an error of 2^-18 crosses few of the 2^-4 steps' borders)
        assert np.mean(codes != f64(y)) <= 2.0 ** -9 + 2 / codes.size, what
    else:
        close(y, want, np.abs(want) * (NORM + HALF[dt]), what)
    for big, fill in ((obig, None if in_place and not q8 else 7.0), (None if ro is None else ro[1], 7.0)):
        if big is not None and fill is not None:
            assert (big[T:].float() == fill).all() and (big[:, D:].float() == fill).all(), f"{what}: outside the rows"
    return y


WIDTHS = [8, 72, 128, 136, 512, 520, 1024, 1032, 2048, 2056, 4096, 4104, 8192, 8200, 16384, 16392, 32768]


@pytest.mark.parametrize("D", WIDTHS)
@pytest.mark.parametrize("T", [1, 5])
def test_norm_widths(T, D):
    check_norm(T, D, "bf16", "bf16", False)
    check_norm(T, D, "bf16", "f32", True, pad=8)
    check_norm(T, D, "f32", "f32", False, pad=4)
    check_norm(T, D, "f32", None, True)
    check_norm(T, D, "bf16", None, False, pad=16)


@pytest.mark.parametrize("T,D", [(513, 1024), (1500, 4096), (700, 264), (5000, 72), (520, 8192), (9000, 128), (70001, 96), (2100, 1544)])
def test_norm_many_rows(T, D):
    """More rows than workgroups, and the forms for many."""
    check_norm(T, D, "bf16", "bf16", True)
    check_norm(T, D, "bf16", "f32", False, in_place=True, pad=8)
    check_norm(T, D, "f32", "f32", True, in_place=True)


@pytest.mark.parametrize("q8", [False, True])
def test_norm_in_place(q8):
    check_norm(3, 640, "bf16", "bf16", q8, in_place=True)
    check_norm(3, 640, "f32", None, q8, in_place=True)


def test_norm_values():
    """Rows of zeros, rows whose 8-bit output would be nothing, large and small ones, a row of one value."""
    x = torch.zeros(6, 64)
    x[1] = 1e-20
    x[2] = rnd(3, 64) * 1e15
    x[3] = rnd(4, 64) * 1e-10
    x[4, 17] = -5.0
    x[5] = 2.0 ** -60
    for io in ("bf16", "f32"):
        check_norm(6, 64, io, None, False, x=x)
        check_norm(6, 64, io, None, True, x=x, eps=1e-2)
    w = torch.ones(64, device=DEV)
    c, s = ssm.rms_norm(torch.zeros(2, 64, device=DEV), w, out_dtype=E4M3)
    assert not c.float().any() and not s.any()
    c, s = ssm.rms_norm(torch.full((1, 64), 1e-38, device=DEV), w, out_dtype=E4M3, eps=1.0)
    assert not c.float().any() and not s.any()  # below 2^-100


@pytest.mark.parametrize("eps", [2.0 ** -126, 1e-30])
def test_norm_smallest_eps(eps):
    """A row of zeros stays zeros, and one beside it is the norm as if eps were none."""
    x = torch.zeros(2, 64)
    x[1] = torch.arange(64) - 31.5
    y = check_norm(2, 64, "f32", None, False, x=x, eps=eps)
    assert np.all(f64(y)[0] == 0)


def test_norm_eps():
    x = rnd(5, 4, 128, scale=0.01)
    a, b = check_norm(4, 128, "f32", None, False, x=x, eps=1e-4), check_norm(4, 128, "f32", None, False, x=x, eps=1e-8)
    assert not torch.equal(a, b)


def test_norm_of_no_tokens():
    w = torch.ones(64, device=DEV)
    x = torch.zeros(0, 64, device=DEV)
    assert ssm.rms_norm(x, w).shape == (0, 64)
    c, s = ssm.rms_norm(x, w, residual=x.clone(), out_dtype=E4M3)
    assert c.shape == (0, 64) and c.dtype == E4M3 and s.shape == (0,)


def test_a_norm_s_rows_are_their_own():
    """A row of NaN leaves the others as they are."""
    w = torch.ones(4096, device=DEV)
    x = rnd(6, 700, 4096).bfloat16().to(DEV)
    want, bad = ssm.rms_norm(x, w), x.clone()
    bad[350] = float("nan")
    got = ssm.rms_norm(bad, w)
    keep = torch.arange(700, device=DEV) != 350
    assert torch.equal(got[keep], want[keep]) and got[350].isnan().all()


def test_norm_past_32_bits():
    """More than 2^32 bytes of rows: the last ones."""
    T, D = 560000, 4096
    x = torch.empty(T, D, dtype=torch.bfloat16, device=DEV)
    x[:8] = 1.0
    tail = rnd(8, 600, D).bfloat16()
    x[-600:] = tail.to(DEV)
    out = torch.empty_like(x)
    ssm.rms_norm(x, torch.ones(D, device=DEV), out=out)
    want = O.rms_norm(f64(tail), np.ones(D), 1e-5)
    close(out[-600:], want, np.abs(want) * (NORM + HALF[torch.bfloat16]), "norm past 32 bits")


# ---------------------------------------------------------------- weights in 4 bits

def special_weights(M, K, io, seed=0):
    """Rows of ordinary values, and groups of ties, zeros, tiny, subnormal and very large ones."""
    w = rnd(seed, M, K) * torch.exp(rnd(seed + 1, M, 1))
    ties = torch.tensor([0.25, -0.75, 1.25, 1.75, -2.5, 3.5, 5.0, -0.25, 4.0, 0.0, -0.0, 6.0, 1.0, 0.2500001, 0.2499999, -5.0])
    w[0, :16] = ties
    if K >= 96:
        w[-1, 32:64] = 0
        w[-1, 64:96] = 2.0 ** -101
        w[0, 64:96] = ties.repeat(2) * 2.0 ** -98
        if M > 2:
            w[1, 32:64] = ties.repeat(2) * 2.0 ** 124
            w[1, 64:96] = 3.3e38
            w[2, :32] = -1e-39
            w[2, 32:64] = torch.linspace(-7, 7, 32)
    return w.to(DT[io])


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("M,K", [(1, 16), (16, 128), (17, 48), (5, 2064), (40, 528), (33, 1040), (130, 272)])
def test_quantize_is_the_definition(M, K, io):
    w = special_weights(M, K, io)
    wv, _ = framed(w, 16, float("nan"))
    q = ssm.q4_quantize(wv)
    codes, scales = O.quantize(f64(w))
    got_c, got_s = O.unpack(q.codes.cpu().numpy(), q.scales.cpu().numpy(), M, K)
    assert np.array_equal(got_s, scales)
    assert np.array_equal(got_c, codes)
    p = ssm.Q4Weight.pack(torch.from_numpy(codes), torch.from_numpy(scales))
    assert torch.equal(q.codes.cpu(), p.codes) and torch.equal(q.scales.cpu(), p.scales)  # what lies past M and K too
    want = O.dequantize(codes, scales)
    for dt in (torch.bfloat16, torch.float32):
        back = ssm.q4_dequantize(q, dtype=dt)
        assert back.shape == (M, K) and np.array_equal(f64(back), want)
        out, big = framed(torch.zeros(M, K, dtype=dt), 16, 7.0)
        ssm.q4_dequantize(q, out=out)
        assert torch.equal(out, back) and (big[M:] == 7).all() and (big[:, K:] == 7).all()


def test_quantize_into_given_buffers():
    w = rnd(1, 50, 160).to(DEV)
    out = ssm.Q4Weight.allocate(50, 160, DEV)
    out.codes.fill_(255), out.scales.fill_(255)
    assert ssm.q4_quantize(w, out=out) is out
    want = ssm.q4_quantize(w)
    assert torch.equal(out.codes, want.codes) and torch.equal(out.scales, want.scales)
    with pytest.raises(ValueError):
        ssm.q4_quantize(w[:49], out=out)


def test_quantizing_a_quantised_weight_keeps_it():
    """Its values are on the grid already, but for groups whose codes stop at 3 or less: those move to a finer one."""
    w = ssm.q4_dequantize(ssm.q4_quantize(rnd(2, 64, 512).to(DEV)), dtype=torch.float32)
    assert torch.equal(ssm.q4_dequantize(ssm.q4_quantize(w), dtype=torch.float32), w)


# ---------------------------------------------------------------- products

def weight(M, K, seed=0, noise=True):
    """A weight of random codes and scales: (packed, values in fp64)."""
    rng = np.random.default_rng(seed)
    c = rng.integers(0, 16, (M, K)).astype(np.uint8)
    s = rng.integers(118, 124, (M, -(-K // 32))).astype(np.uint8)
    w = ssm.Q4Weight.pack(torch.from_numpy(c), torch.from_numpy(s))
    if noise and M % 16:  # past the last row anything may lie
        w.codes[-1].view(-1, 4, 16, 16)[:, :, M % 16:] = 0x5F
        w.scales[-1].view(-1, 4, 16, 4)[:, :, M % 16:] = 255
    return ssm.Q4Weight(w.codes.to(DEV), w.scales.to(DEV), M, K), O.dequantize(c, s)


def tokens(T, K, kind, seed=0):
    """(tokens, scales or None, values in fp64)."""
    x = rnd(seed, T, K)
    if kind != "e4m3":
        x = x.to(DT[kind])
        return x, None, f64(x)
    s = torch.rand(T, generator=torch.Generator().manual_seed(seed + 1)) + 0.5
    x = (x * 100).clamp(-448, 448).to(E4M3)
    return x, s.to(DEV), f64(x) * f64(s)[:, None]


LINEAR = [(1, 1, 16), (1, 16, 128), (1, 17, 144), (3, 1000, 1552), (2, 40, 512), (16, 33, 528), (16, 288, 4112), (17, 1, 16),
          (17, 129, 144), (31, 128, 640), (32, 300, 2064), (33, 65, 528), (64, 384, 1040), (65, 200, 272), (100, 2048, 2048),
          (127, 130, 400), (128, 128, 128), (129, 257, 1552), (300, 520, 656), (1000, 96, 80)]


def check_linear(T, M, K, kind, out_dtype, seed=0):
    w, wv = weight(M, K, seed)
    x, xs, xf = tokens(T, K, kind, seed + 5)
    xv, _ = framed(x, 16, float("nan"))
    out, big = framed(torch.zeros(T, M, dtype=out_dtype), 5, 7.0)
    got = ssm.q4_linear(xv, w, x_scale=xs, out=out)
    assert got is out
    what = f"linear {T}x{M}x{K} {kind} {out_dtype}"
    want, mags = xf @ wv.T, np.abs(xf) @ np.abs(wv).T
    coded = 2.0 ** -10 if kind == "e4m3" and out_dtype == torch.bfloat16 else 0.0
    close(got, want, (K * 2.0 ** -23 + coded) * mags + HALF[out_dtype] * np.abs(want) + 1e-30, what)
    err = np.linalg.norm(f64(got) - want) / max(np.linalg.norm(want), 1e-30)
    print(what, "error as a whole", err)
    assert err <= HALF[out_dtype] + 2.0 ** -23 * max(K / 2, 1) ** 0.5 + 2.0 ** -23, f"{what}: {err:.2e} as a whole"
    assert (big[T:] == 7).all() and (big[:, M:] == 7).all(), f"{what}: outside the rows"
    again = ssm.q4_linear(xv, w, x_scale=xs, out_dtype=out_dtype)
    assert again.dtype == out_dtype and torch.equal(again, got), f"{what}: another result"


@pytest.mark.parametrize("kind", ["bf16", "f32", "e4m3"])
@pytest.mark.parametrize("T,M,K", LINEAR)
def test_linear(T, M, K, kind):
    check_linear(T, M, K, kind, torch.float32)
    check_linear(T, M, K, kind, torch.bfloat16, seed=1)


# Sizes that reach each form of the calls of few tokens (rows of a workgroup) and of tiles (how many there are).
FORMS = [(1, 9000, 144), (4, 8209, 656), (12, 5000, 400), (16, 9000, 144), (20, 5000, 144), (32, 8300, 528), (300, 1000, 2064),
         (520, 1000, 2064), (1000, 1100, 2064), (1030, 2100, 1552), (2050, 2100, 1040), (2100, 2101, 400), (3000, 3100, 528),
         (91, 28001, 272), (600, 3900, 1040), (1510, 4090, 272), (1010, 4001, 272), (1300, 4095, 400),
         (2040, 4090, 272), (2200, 4090, 144), (4100, 3200, 400)]


@pytest.mark.parametrize("kind", ["bf16", "f32", "e4m3"])
@pytest.mark.parametrize("T,M,K", FORMS)
def test_linear_forms(T, M, K, kind):
    check_linear(T, M, K, kind, torch.bfloat16)
    check_linear(T, M, K, kind, torch.float32, seed=1)


@pytest.mark.parametrize("kind", ["bf16", "f32", "e4m3"])
@pytest.mark.parametrize("T,M,K", [(7, 4100, 656), (5, 20005, 400), (32, 20000, 1168), (24, 12003, 528), (17, 34000, 272), (32, 33001, 1040),
                                   (40, 33000, 272), (64, 32790, 912), (64, 66001, 144)])
def test_linear_few_tokens_by_many_rows(T, M, K, kind):
    """Up to 32 and up to 64 tokens have tiles of their own where there are more rows than CUs take at once."""
    check_linear(T, M, K, kind, torch.bfloat16)
    check_linear(T, M, K, kind, torch.float32, seed=1)


@pytest.mark.parametrize("kind", ["bf16", "f32", "e4m3"])
@pytest.mark.parametrize("T", [1, 7, 16, 17, 40, 64, 150])
def test_linear_by_the_identity_gives_the_tokens(T, kind):
    """Every value comes back from its own place, with all its bits (fp32: in three parts)."""
    K = 272
    c = torch.zeros(K, K, dtype=torch.uint8)
    c[torch.arange(K), torch.arange(K)] = 2  # 1.0
    w = ssm.Q4Weight.pack(c, torch.full((K, -(-K // 32)), 127, dtype=torch.uint8))
    w = ssm.Q4Weight(w.codes.to(DEV), w.scales.to(DEV), K, K)
    x, xs, xf = tokens(T, K, kind)
    got = ssm.q4_linear(x.to(DEV), w, x_scale=xs, out_dtype=torch.float32)
    want = x.float() if xs is None else x.float() * xs.cpu()[:, None]
    assert torch.equal(got.cpu(), want)


@pytest.mark.parametrize("kind", ["bf16", "f32", "e4m3"])
@pytest.mark.parametrize("T", [3, 40, 130])
@pytest.mark.parametrize("lo,hi", [(117, 137), (123, 133)])
def test_linear_takes_every_group_s_scale(T, kind, lo, hi):
    """All ones times codes of one: a row's sum is the sum of its groups' scales."""
    M, K = 100, 1104
    rng = np.random.default_rng(3)
    s = rng.integers(lo, hi, (M, -(-K // 32))).astype(np.uint8)
    w = ssm.Q4Weight.pack(torch.full((M, K), 2, dtype=torch.uint8), torch.from_numpy(s))
    w = ssm.Q4Weight(w.codes.to(DEV), w.scales.to(DEV), M, K)
    xs = torch.ones(T, device=DEV) if kind == "e4m3" else None
    got = f64(ssm.q4_linear(torch.ones(T, K, device=DEV).to(DT[kind]), w, x_scale=xs, out_dtype=torch.float32))
    want = O.dequantize(np.full((M, K), 2), s).sum(1)
    # Scales of 2^-4 .. 2^5: sums are below 2^5 1104 < 2^16 in steps of 2^-4, exact in fp32's 24 bits.  Of 2^-10 .. 2^9 they
    # take up to 30: each of at most 1104 additions of positive terms rounds by 2^-23 of the sum at most.
    tol = 0.0 if lo == 123 else 1104 * 2.0 ** -23
    assert got.shape == (T, M) and np.all(np.abs(got - want) <= tol * want)


@pytest.mark.parametrize("T", [3, 40, 130])
def test_what_the_instruction_on_codes_keeps(T):
    """Of eight columns' products what is at least 2^-13 of the largest; an fp32 output keeps all."""
    K = 128
    c = torch.zeros(8, K, dtype=torch.uint8)
    c[:, 0], c[:, 3] = 7, 1      # 6 and 0.5
    c[4:, 40] = 15               # -6: what is left of the sum
    w = ssm.Q4Weight.pack(c, torch.full((8, 4), 127, dtype=torch.uint8))
    w = ssm.Q4Weight(w.codes.to(DEV), w.scales.to(DEV), 8, K)
    x = torch.zeros(T, K, device=DEV)
    x[:, 0] = x[:, 40] = 256
    for small in (0.25, 2.0 ** -9):  # products of 1536 (2^10.6) and 2^-3 or 2^-10, which is 2^-13 of 2^10 or less
        x[:, 3] = small
        one = torch.ones(T, device=DEV)
        exact = ssm.q4_linear(x.to(E4M3), w, x_scale=one, out_dtype=torch.float32)
        assert (exact[:, :4] == 1536 + small / 2).all() and (exact[:, 4:] == small / 2).all()
        bf = ssm.q4_linear(x.to(E4M3), w, x_scale=one)
        assert ((bf[:, 4:].float() - small / 2).abs() <= 1536 * 2.0 ** -13).all()


@pytest.mark.parametrize("T", [16, 64, 200])
def test_a_token_s_values_stay_with_it(T):
    w, _ = weight(200, 528)
    x = rnd(1, T, 528).bfloat16().to(DEV)
    want, bad = ssm.q4_linear(x, w), x.clone()
    bad[T // 2] = float("nan")
    got = ssm.q4_linear(bad, w)
    keep = torch.arange(T, device=DEV) != T // 2
    assert torch.equal(got[keep], want[keep]) and got[T // 2].isnan().all()


def test_linear_of_no_tokens():
    w, _ = weight(40, 64)
    assert ssm.q4_linear(torch.zeros(0, 64, device=DEV), w).shape == (0, 40)
    got = ssm.q4_linear(torch.zeros(0, 64, device=DEV).to(E4M3), w, x_scale=torch.zeros(0, device=DEV))
    assert got.shape == (0, 40) and got.dtype == torch.bfloat16


def test_linear_past_32_bits():
    """More than 2^32 bytes of codes: the last rows, for few tokens and for more; then of tokens."""
    M, K = 1 << 20, 8720
    w = ssm.Q4Weight.allocate(M, K, DEV)
    w.codes.zero_(), w.scales.fill_(127)
    last, wv = weight(160, K, noise=False)
    w.codes[-10:] = last.codes
    w.scales[-10:] = last.scales
    for T in (2, 20, 40):
        x = rnd(T, T, K).bfloat16()
        got = ssm.q4_linear(x.to(DEV), w, out_dtype=torch.float32)
        assert not got[:, :M - 160].any()
        want, mags = f64(x) @ wv.T, np.abs(f64(x)) @ np.abs(wv).T
        close(got[:, -160:], want, K * 2.0 ** -23 * mags, f"past 32 bits, {T} tokens")
    del w, got
    T, M, K = 600000, 24, 4096
    w, wv = weight(M, K)
    for kind in ("bf16", "e4m3"):
        x, xs, xf = tokens(500, K, kind)
        big = torch.zeros(T if kind == "bf16" else 2 * T, K, device=DEV, dtype=torch.bfloat16 if kind == "bf16" else torch.uint8).view(x.dtype)
        big.view(torch.uint8)[-500:] = x.view(torch.uint8).view(500, -1).to(DEV)
        scale = None if xs is None else torch.cat([torch.ones(len(big) - 500, device=DEV), xs])
        got = ssm.q4_linear(big, w, x_scale=scale, out_dtype=torch.float32)
        want, mags = xf @ wv.T, np.abs(xf) @ np.abs(wv).T
        assert not got[:-500].any()
        close(got[-500:], want, K * 2.0 ** -23 * mags, f"past 32 bits of tokens, {kind}")


def test_quantize_past_32_bits():
    """More than 2^32 bytes of a weight: the last rows, made and read back."""
    M, K = 560000, 4096
    w = torch.zeros(M, K, dtype=torch.bfloat16, device=DEV)
    tail = rnd(1, 320, K).bfloat16().to(DEV)
    w[-320:] = tail
    q, t = ssm.q4_quantize(w), ssm.q4_quantize(tail)
    assert torch.equal(q.codes[-20:], t.codes) and torch.equal(q.scales[-20:], t.scales) and not q.codes[:-20].any()
    w.fill_(1)
    ssm.q4_dequantize(q, out=w)
    assert torch.equal(w[-320:], ssm.q4_dequantize(t)) and not w[:-320].any()


# ---------------------------------------------------------------- as they are used together, and how they are called

def pipeline(T=24, D=1040, M=600):
    w, wv = weight(M, D, seed=9)
    return dict(x=rnd(1, T, D).bfloat16().to(DEV), res=rnd(2, T, D).to(DEV), g=(1 + 0.1 * rnd(3, D)).to(DEV), w=w, wv=wv)


def step(p, **kw):
    codes, scale = ssm.rms_norm(p["x"], p["g"], residual=p["res"], out_dtype=E4M3, **kw)
    return codes, scale, ssm.q4_linear(codes, p["w"], x_scale=scale, **kw)


@pytest.mark.parametrize("T", [1, 24, 70])
def test_a_block_s_way_in(T):
    """The stream, its norm in 8 bits and the projection of it."""
    p = pipeline(T)
    h = p["x"].float() + p["res"]
    codes, scale, y = step(p)
    assert torch.equal(p["res"], h)
    want = (f64(codes) * f64(scale)[:, None]) @ p["wv"].T
    mags = np.abs(f64(codes) * f64(scale)[:, None]) @ np.abs(p["wv"]).T
    close(y, want, (1040 * 2.0 ** -23 + 2.0 ** -10) * mags + 2.0 ** -8 * np.abs(want), "a block's way in")
    # against the definitions without the 8 bits: each code is within 2^-4 of its value, errors of independent signs
    full = O.rms_norm(f64(h), f64(p["g"]), 1e-5) @ p["wv"].T
    assert np.linalg.norm(f64(y) - full) <= 2.0 ** -4 * np.linalg.norm(full)


@pytest.mark.parametrize("native", [True, False])
def test_calls_on_another_stream(native, monkeypatch):
    if not native:
        monkeypatch.setattr(B, "_native", B._NoNative)
    want = [t.clone() for t in step(pipeline(70))]
    s = torch.cuda.Stream()
    p = pipeline(70)
    torch.cuda.synchronize()
    got = step(p, stream=s)
    s.synchronize()
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got, want))
    p = pipeline(70)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        got = step(p)
    s.synchronize()
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got, want))


def test_the_native_half_takes_the_usual_calls_and_gives_the_same(monkeypatch):
    p = pipeline(70)
    fast = B._bound()
    assert fast is not B._NoNative
    seen = []

    class Spy:
        def __getattr__(self, name):
            def call(*a):
                seen.append(getattr(fast, name)(*a))
                return seen[-1]
            return call
    monkeypatch.setattr(B, "_native", Spy())

    def calls():
        x, g, w = p["x"], p["g"], p["w"]
        res = p["res"].clone()
        out = [ssm.rms_norm(x, g), ssm.rms_norm(x.float(), g), *ssm.rms_norm(x, g, residual=res, out_dtype=E4M3), res]
        ro = torch.zeros_like(res)
        out += [ssm.rms_norm(x, g, residual=res, residual_out=ro, eps=0.5), ro, ssm.rms_norm(x, g, out=torch.zeros_like(x))]
        c, s = torch.zeros_like(x, dtype=E4M3), torch.zeros(70, device=DEV)
        out += [*ssm.rms_norm(x, g, out=c, scale=s)]
        out += [ssm.q4_linear(x, w), ssm.q4_linear(x, w, out_dtype=torch.float32), ssm.q4_linear(x.float(), w),
                ssm.q4_linear(c, w, x_scale=s), ssm.q4_linear(x[:3], w, out=torch.zeros(3, 600, device=DEV))]
        q, r = ssm.q4_quantize(x), ssm.q4_quantize(x.float())
        assert isinstance(q, ssm.Q4Weight) and q.shape == x.shape
        out += [q.codes, q.scales, r.codes, r.scales, ssm.q4_dequantize(q), ssm.q4_dequantize(q, dtype=torch.float32),
                ssm.q4_dequantize(r, out=torch.zeros_like(x))]
        return out
    a = calls()
    assert len(seen) == 16 and all(r is not NotImplemented for r in seen)
    monkeypatch.setattr(B, "_native", B._NoNative)
    for u, v in zip(a, calls()):
        assert u.dtype == v.dtype and torch.equal(u.reshape(-1).view(torch.uint8), v.reshape(-1).view(torch.uint8))


def test_refusals_on_the_gpu_are_worded():
    p = pipeline()
    x, g, w = p["x"], p["g"], p["w"]
    for what, call in (
            ("weight", lambda: ssm.rms_norm(x, g[:-1])), ("weight", lambda: ssm.rms_norm(x, g.bfloat16())),
            ("residual", lambda: ssm.rms_norm(x, g, residual=p["res"][1:])), ("out", lambda: ssm.rms_norm(x, g, out=x[1:])),
            ("contiguous", lambda: ssm.rms_norm(x[:, ::2], g[::2].contiguous())),
            ("x: shape", lambda: ssm.q4_linear(x[:, :-16], w)), ("x_scale", lambda: ssm.q4_linear(x.to(E4M3), w)),
            ("x_scale", lambda: ssm.q4_linear(x, w, x_scale=torch.ones(24, device=DEV))),
            ("x_scale", lambda: ssm.q4_linear(x.to(E4M3), w, x_scale=torch.ones(23, device=DEV))),
            ("codes", lambda: ssm.q4_linear(x, w._replace(codes=w.codes[1:]))),
            ("scales", lambda: ssm.q4_linear(x, w._replace(scales=w.scales.int()))),
            ("codes", lambda: ssm.q4_dequantize(w._replace(codes=w.codes[1:]))),
            ("out: shape", lambda: ssm.q4_dequantize(w, out=torch.zeros(3, 1040, device=DEV))),
            ("multiple of 16", lambda: ssm.q4_quantize(torch.zeros(4, 24, device=DEV))),
            ("contiguous", lambda: ssm.q4_quantize(torch.zeros(4, 64, device=DEV)[:, ::2])),
            ("4-bit weight", lambda: ssm.q4_linear(x, w._replace(in_features=1041)))):
        with pytest.raises(ValueError, match=what):
            call()
    with pytest.raises(TypeError):
        ssm.rms_norm(x, g, residual=p["res"].half())
    with pytest.raises(TypeError):
        ssm.rms_norm(x.float(), g, residual=x)  # a residual of less precision than the tokens
    for call in (lambda: ssm.rms_norm(x, g, eps=0.0), lambda: ssm.rms_norm(x, g, residual=x, out=x),
                 lambda: ssm.rms_norm(x[:, 4:1004], g[:1000].contiguous())):
        with pytest.raises(ssm.SsmError):
            call()


def test_captured_calls_replay():
    """A captured block's way in, replayed with new tokens between eager calls of the same operators; two graphs with
    memory of their own, replayed in turn."""
    ps = [pipeline(40), pipeline(40)]
    for p in ps:
        p["res"].zero_()
    torch.cuda.synchronize()
    graphs = []
    side = torch.cuda.Stream()
    for p in ps:
        with torch.cuda.stream(side):
            step(p)
        side.synchronize()
        p["res"].zero_()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = step(p)
        graphs.append((graph, p, got))
    for k in range(4):
        for i, (graph, p, got) in enumerate(graphs):
            x = rnd(100 + 10 * k + i, *p["x"].shape).bfloat16().to(DEV)
            p["x"].copy_(x)
            p["res"].fill_(0.25 * k)
            graph.replay()
        torch.cuda.synchronize()
        for i, (graph, p, got) in enumerate(graphs):
            eager = dict(p, res=torch.full_like(p["res"], 0.25 * k))
            want = step(eager)
            assert torch.equal(eager["res"], p["res"])
            for a, b in zip(got, want):
                assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), (k, i)
