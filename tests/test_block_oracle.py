"""oracle/block.py pinned by other means, planted mistakes that the pins must notice, and Q4Weight.pack against the layout
(no GPU)."""
import numpy as np
import pytest
import torch

import selective_state_space_causal_amd as ssm
from oracle import block as O

RNG = np.random.default_rng(7)


def test_norm_has_unit_mean_square_and_no_scale():
    h = RNG.standard_normal((5, 40)) * 3
    y = O.rms_norm(h, np.ones(40), 1e-12)
    assert np.allclose((y * y).mean(-1), 1) and np.allclose(O.rms_norm(7 * h, np.ones(40), 1e-12), y)
    w = RNG.standard_normal(40)
    assert np.allclose(O.rms_norm(h, w, 1e-12), y * w)
    t = torch.nn.functional.rms_norm(torch.from_numpy(h), (40,), torch.from_numpy(w), 0.5).numpy()
    assert np.allclose(O.rms_norm(h, w, 0.5), t)
    assert not np.allclose(O.rms_norm(h, w, 0.25), t)  # eps forgotten, or outside the root
    assert not np.allclose(O.rms_norm(h - h.mean(-1, keepdims=True), w, 0.5), t)  # the mean taken off, as another norm does


def test_row_codes_are_torch_s():
    y = RNG.standard_normal((20, 64)).astype(np.float32)
    c, s = O.row_codes(y)
    t = torch.from_numpy(y).double()
    want = (t * (448 / t.abs().amax(-1, keepdim=True))).to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(c, want) and np.allclose(s, np.abs(y).max(-1) / 448)
    assert np.abs(c).max() == 448 and np.abs(c * s[:, None] - y).max() <= 16 * s.max()
    z, sz = O.row_codes(np.full((1, 8), 2.0 ** -101))
    assert not z.any() and not sz.any()


@pytest.mark.parametrize("amax,e", [(6.0, 127), (4.0, 127), (6.99, 127), (7.0, 128), (3.5, 127), (3.49, 126), (1.0, 125), (2.0 ** -100, 25),
                                    (3.4e38, 252)])
def test_scale_brings_the_largest_to_four_to_six(amax, e):
    w = np.zeros((1, 32))
    w[0, 5] = -amax
    c, s = O.quantize(w)
    assert s[0, 0] == e
    v = O.dequantize(c, s)[0, 5]
    assert v < 0 and c[0, 5] >= 8 and np.count_nonzero(c) == 1
    if e < 252:
        assert abs(v + amax) <= amax / 7 + 1e-12  # 6.99 is held as 6


def test_codes_are_the_nearest_with_ties_to_even():
    # a group of largest value 4: scale 1
    x = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 0.26, 0.24, 0.74, 1.76, 2.51, 3.49, -0.25, -0.75, -1.25, -2.5, 4.0] + [0.0] * 15)
    c, s = O.quantize(x[None])
    assert s[0, 0] == 127
    want = [0, 1, 1, 2, 2, 4, 0.5, 0, 0.5, 2, 3, 3, 0, -1, -1, -2, 4]
    assert np.array_equal(O.dequantize(c, s)[0, :17], want)
    away = [0.5, 1, 1.5, 2, 3, 4]  # ties away from zero would give these
    assert want[:6] != away
    assert c[0, 12] == 8  # what rounds to zero keeps its sign


def test_tiny_groups_are_zeros():
    w = np.full((1, 48), 2.0 ** -100 * 0.99)
    w[0, 32:] = -1.0
    c, s = O.quantize(w)
    assert not c[0, :32].any() and s[0, 0] == 127 and s[0, 1] == 125 and (c[0, 32:] == 14).all()


@pytest.mark.parametrize("M,K", [(1, 16), (17, 48), (33, 528), (16, 128), (40, 1040)])
def test_pack_lays_codes_out_as_documented(M, K):
    c = RNG.integers(0, 16, (M, K)).astype(np.uint8)
    s = RNG.integers(2, 253, (M, -(-K // 32))).astype(np.uint8)
    w = ssm.Q4Weight.pack(torch.from_numpy(c), torch.from_numpy(s))
    assert w.shape == (M, K) and w.codes.is_contiguous() and w.scales.is_contiguous()
    uc, us = O.unpack(w.codes.numpy(), w.scales.numpy(), M, K)
    assert np.array_equal(uc, c) and np.array_equal(us, s)
    assert w.codes.numel() == -(-M // 16) * -(-K // 128) * 1024 and w.scales.numel() == -(-M // 16) * -(-K // 512) * 256
    assert int(w.codes.int().sum()) == int((c[:, ::2].astype(int) + 16 * c[:, 1::2]).sum())  # zeros past M and K
    wrong = w.codes.numpy().copy()
    wrong = wrong.reshape(*wrong.shape[:2], 4, 16, 16).swapaxes(2, 3).reshape(wrong.shape)  # rows and groups exchanged
    assert M == 1 or not np.array_equal(O.unpack(wrong, w.scales.numpy(), M, K)[0], c)


def test_pack_refuses():
    c, s = torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(4, 1, dtype=torch.uint8)
    for bad_c, bad_s in ((c[0], s), (c.int(), s), (c, s.int()), (c, s[:3]), (c[:, :24], s), (c[:, :0], s[:, :0])):
        with pytest.raises(ValueError):
            ssm.Q4Weight.pack(bad_c, bad_s)
    with pytest.raises(ValueError):
        ssm.Q4Weight.allocate(0, 16, device="cpu")
    with pytest.raises(ValueError):
        ssm.Q4Weight.allocate(2 ** 20, 2 ** 20, device="cpu")
