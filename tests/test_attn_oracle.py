"""oracle/attn.py pinned by other means (complex rotation, brute-force softmax sums, torch's own e4m3
conversion), and planted mistakes that the pins must notice."""
import math

import numpy as np
import pytest
import torch

from oracle import attn as O

RNG = np.random.default_rng(3)


def rope_by_complex(x, pos, freq, inter, ms):
    h = len(freq)
    out = np.array(x)
    for t in range(x.shape[0]):
        for i in range(h):
            a, b = (2 * i, 2 * i + 1) if inter else (i, i + h)
            z = (x[t, :, a] + 1j * x[t, :, b]) * ms * np.exp(1j * pos[t] * freq[i])
            out[t, :, a], out[t, :, b] = z.real, z.imag
    return out


@pytest.mark.parametrize("inter", [False, True])
def test_rope_is_a_complex_product(inter):
    x = RNG.standard_normal((5, 2, 12))
    pos, freq = np.array([0, 1, 7, 100, 3]), np.array([1.0, 0.3, 0.01, 0.5])
    want = rope_by_complex(x, pos, freq, inter, 1.5)
    assert np.allclose(O.rope(x, pos, freq, inter, 1.5), want, atol=1e-12)
    assert not np.allclose(O.rope(x, pos, freq, not inter, 1.5), want, atol=1e-3)   # the other layout
    assert not np.allclose(O.rope(x, -pos, freq, inter, 1.5), want, atol=1e-3)      # the other way round
    assert not np.allclose(O.rope(x, pos, freq, inter, 1.0), want, atol=1e-3)       # the factor forgotten


def test_rope_keeps_products_of_equal_distance():
    q, k, f = RNG.standard_normal((1, 1, 8)), RNG.standard_normal((1, 1, 8)), np.array([1.0, 0.1, 0.02, 0.003])
    dot = lambda i, j: float((O.rope(q, [i], f, False, 1.0) * O.rope(k, [j], f, False, 1.0)).sum())  # noqa: E731
    assert abs(dot(9, 2) - dot(1007, 1000)) < 1e-9 and abs(dot(9, 2) - dot(9, 3)) > 1e-3


def test_e4m3_is_torch_s():
    x = torch.cat([torch.randn(20000) * 10.0 ** e for e in (-3, -2, -1, 0, 1, 2)]).clamp(-448, 448)
    assert np.array_equal(O.to_e4m3(x.numpy()), x.to(torch.float8_e4m3fn).double().numpy())
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    v = codes[~codes.isnan()].numpy()
    assert np.array_equal(O.to_e4m3(v), v)
    mid = (O.E4M3[1:] + O.E4M3[:-1]) / 2  # ties, exact in fp32
    assert np.array_equal(O.to_e4m3(mid), torch.tensor(mid).float().to(torch.float8_e4m3fn).double().numpy())


@pytest.mark.parametrize("kind,step", [("int8", None), ("e4m3", None)])
def test_quantize(kind, step):
    x = RNG.standard_normal((50, 64)).astype(np.float32) * 3
    x[0] = 0
    x[1] = 2.0 ** -120
    x[2] = 1e30
    code, s = O.quantize(x, kind)
    top = 127 if kind == "int8" else 448
    assert np.abs(code).max() == top and s[0] == 0 and s[1] == 0 and np.all(code[:2] == 0)
    val = code * s[:, None].astype(np.float64)
    # half a step: of the row's scale for int8, of the value (2^-4) or the smallest code (2^-10) for e4m3; the scale's own
    # rounding and the multiplier's add 2^-22
    half = 0.5 * s[:, None] if kind == "int8" else np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * s[:, None])
    assert np.all(np.abs(val - x)[2:] <= (half + 2.0 ** -22 * np.abs(x))[2:])


def test_attend_by_sums():
    H, D, n = 3, 8, 11
    q, k, v = RNG.standard_normal((H, D)), RNG.standard_normal((n, D)), RNG.standard_normal((n, D))
    for seen in (1, 5, n):
        out, lse, mag, smax, _ = O.attend(q, k, v, 0.7, seen)
        for h in range(H):
            w = [math.exp(0.7 * float(q[h] @ k[j])) for j in range(seen)]
            assert np.allclose(out[h], sum(w[j] * v[j] for j in range(seen)) / sum(w))
            assert np.allclose(mag[h], sum(w[j] * np.abs(v[j]) for j in range(seen)) / sum(w))
            assert abs(lse[h] - math.log(sum(w))) < 1e-12
    out, lse, *_ = O.attend(q, k, v, 0.7, 0)
    assert np.all(out == 0) and np.all(np.isneginf(lse))


def test_prefill_masks_and_heads():
    q, k, v = RNG.standard_normal((7, 4, 8)), RNG.standard_normal((9, 2, 8)), RNG.standard_normal((9, 2, 8))
    cu_q, cu_k = [0, 3, 3, 7], [0, 6, 7, 9]
    out = O.prefill(q, k, v, cu_q, cu_k, True, 0.5)[0]
    # token 1 of sequence 0 (3 queries, 6 keys) sees keys 0..4; head 3 reads key head 1
    assert np.allclose(out[1, 3], O.attend(q[1, 3:4], k[:5, 1], v[:5, 1], 0.5, 5)[0][0])
    # sequence 2: 4 queries, 2 keys; its first two see nothing, its third one key
    assert np.all(out[3:5] == 0) and np.allclose(out[5, 0], v[7, 0]) and np.all(out[6] != 0)
    full = O.prefill(q, k, v, cu_q, cu_k, False, 0.5)[0]
    assert np.allclose(full[0, 0], O.attend(q[0, :1], k[:6, 0], v[:6, 0], 0.5, 6)[0][0])


def test_decode_follows_the_table():
    pages, Hkv, page, D = 5, 2, 16, 8
    k, v = RNG.standard_normal((pages, Hkv, page, D)), RNG.standard_normal((pages, Hkv, page, D))
    q = RNG.standard_normal((2, 4, D))
    table = np.array([[3, 0, 9], [-1, 4, 2]])
    out = O.decode(q, k, v, table, [20, 18], 0.5)[0]
    kk = np.concatenate([k[3, 1], k[0, 1, :4]])
    vv = np.concatenate([v[3, 1], v[0, 1, :4]])
    assert np.allclose(out[0, 2], O.attend(q[0, 2:3], kk, vv, 0.5, 20)[0][0])
    assert np.allclose(out[1, 0], O.attend(q[1, :1], k[4, 0, :2], v[4, 0, :2], 0.5, 2)[0][0])  # page -1 is not seen


def test_tolerance_notices_mistakes():
    """A dropped key, a wrong head or an unscaled product is far outside the tolerance that the GPU tests use."""
    q, k, v = RNG.standard_normal((4, 2, 64)), RNG.standard_normal((40, 1, 64)), RNG.standard_normal((40, 1, 64))
    ref = O.prefill(q, k, v, [0, 4], [0, 40], True, 0.125)
    tol, ltol = O.attention_tolerance(2.0 ** -8, 2.0 ** -8, *ref[:1], *ref[2:], 64, 1024)
    for bad in (O.prefill(q, k, v, [0, 4], [0, 39], True, 0.125), O.prefill(q[:, ::-1], k, v, [0, 4], [0, 40], True, 0.125),
                O.prefill(q, k, v, [0, 4], [0, 40], False, 0.125), O.prefill(q, k, v, [0, 4], [0, 40], True, 1.0)):
        assert np.any(np.abs(bad[0] - ref[0]) > tol)
        assert np.any(np.abs(bad[1] - ref[1]) > ltol)
