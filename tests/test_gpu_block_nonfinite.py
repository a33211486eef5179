"""NaN and infinities in the operators that store 8 or 4 bits.  Rows of the 8-bit norm that hold one read back as NaN, as by the
definition (the row's largest magnitude, and with it its scale, is NaN), and do not turn into plausible numbers on the way through a
4-bit product; other rows are as without them.  Likewise the groups of a weight in 4 bits."""
import pytest
import torch

import selective_state_space_causal_amd as ssm

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
E4M3 = torch.float8_e4m3fn
NAN, INF = float("nan"), float("inf")


def rnd(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed))


def values(codes, scale):
    return codes.float() * scale[:, None]


# Widths that reach each form: threads to a row, pieces to a thread.
@pytest.mark.parametrize("D", [64, 264, 1040, 4096, 8192, 8208, 32768])
@pytest.mark.parametrize("io,res", [("bf16", None), ("bf16", "f32"), ("f32", None), ("f32", "f32"), ("bf16", "bf16")])
@pytest.mark.parametrize("bad", [NAN, INF, -INF])
def test_a_row_that_is_not_finite_reads_back_as_nan(D, io, res, bad):
    T, types = 9, {"bf16": torch.bfloat16, "f32": torch.float32}
    w = (1 + 0.1 * rnd(1, D)).to(DEV)
    x = rnd(2, T, D).to(types[io]).to(DEV)
    r = None if res is None else rnd(3, T, D).to(types[res]).to(DEV)
    rows, places = [0, 4, 8], [0, D // 2 + 1, D - 1]
    xb, rb = x.clone(), None if r is None else r.clone()
    for row, place in zip(rows, places):
        (xb if row != 4 or rb is None else rb)[row, place] = bad
    want = ssm.rms_norm(x, w, residual=None if r is None else r.clone(), out_dtype=E4M3)
    got = ssm.rms_norm(xb, w, residual=rb, out_dtype=E4M3)
    keep = [i for i in range(T) if i not in rows]
    assert torch.equal(got[0][keep].view(torch.uint8), want[0][keep].view(torch.uint8)) and torch.equal(got[1][keep], want[1][keep])
    assert values(*got)[rows].isnan().all()
    if D % 16:
        return  # no 4-bit weight has such rows
    q = ssm.q4_quantize(rnd(4, 48, D).to(DEV))
    for dt in (torch.bfloat16, torch.float32):
        y, y0 = (ssm.q4_linear(c, q, x_scale=s, out_dtype=dt) for c, s in (got, want))
        assert y[rows].isnan().all() and torch.equal(y[keep], y0[keep])


@pytest.mark.parametrize("D", [64, 4096, 8208])
def test_a_row_of_zeros_with_one_nan(D):
    """Nothing else in the row: its largest magnitude without the NaN is zero."""
    x = torch.zeros(3, D, device=DEV)
    x[1, 5] = NAN
    c, s = ssm.rms_norm(x, torch.ones(D, device=DEV), out_dtype=E4M3)
    v = values(c, s)
    assert v[1].isnan().all() and not v[0].any() and not v[2].any()


@pytest.mark.parametrize("D", [64, 4096, 8208])
def test_a_weight_that_is_nan_stays_in_its_column(D):
    x, w = rnd(1, 5, D).bfloat16().to(DEV), torch.ones(D, device=DEV)
    w[7] = 0
    want = values(*ssm.rms_norm(x, w, out_dtype=E4M3))
    w[7] = NAN
    got = values(*ssm.rms_norm(x, w, out_dtype=E4M3))
    keep = torch.arange(D, device=DEV) != 7
    assert got[:, 7].isnan().all() and torch.equal(got[:, keep], want[:, keep])


@pytest.mark.parametrize("io", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,K", [(1, 16), (5, 48), (40, 1040)])
@pytest.mark.parametrize("bad", [NAN, INF, -INF])
def test_a_group_of_a_weight_that_is_not_finite_reads_back_as_nan(M, K, io, bad):
    """4 bits hold no NaN or infinity: the group's scale does, and a product with its row is NaN."""
    w = rnd(1, M, K).to(io).to(DEV)
    want, wb = ssm.q4_quantize(w), w.clone()
    rows = sorted({0, M // 2, M - 1})
    places = [(5 + 37 * i) % K for i in rows]
    for row, place in zip(rows, places):
        wb[row, place] = bad
    q = ssm.q4_quantize(wb)
    gone = torch.zeros(M, K, dtype=torch.bool, device=DEV)
    for row, place in zip(rows, places):
        gone[row, place // 32 * 32:place // 32 * 32 + 32] = True
    for dt in (torch.bfloat16, torch.float32):
        a, b = ssm.q4_dequantize(q, dtype=dt), ssm.q4_dequantize(want, dtype=dt)
        assert a[gone].isnan().all() and torch.equal(a[~gone], b[~gone])
    keep = [m for m in range(M) if m not in rows]
    for T in (1, 3, 7, 20, 40, 130):
        x = rnd(T, T, K).to(DEV)
        for xt, xs in ((x, None), (x.bfloat16(), None), (x.to(E4M3), torch.ones(T, device=DEV))):
            y, y0 = (ssm.q4_linear(xt, v, x_scale=xs) for v in (q, want))
            assert y[:, rows].isnan().all() and torch.equal(y[:, keep], y0[:, keep])
