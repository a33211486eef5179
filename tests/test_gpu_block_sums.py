"""Products of 8-bit tokens where a few columns are far larger than the rest and cancel: what a row of activations with outlier
channels gives.  Every product is a multiple of 2^-5 and every partial sum of them, in any order, is below 2^18 in magnitude, so
sums in fp32 are exact: an fp32 output equals the definition, and a bf16 one its rounding."""
import numpy as np
import pytest
import torch

import selective_state_space_causal_amd as ssm
from oracle import block as O

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
E4M3 = torch.float8_e4m3fn


def outliers(T, M, K, seed=0):
    """(tokens, weight on the device, their product in fp64): pairs of columns of 448 whose weights are equal and opposite,
    among tokens of sixteenths up to 1; scales of 1."""
    rng = np.random.default_rng(seed)
    x = rng.integers(-16, 17, (T, K)) / 16.0
    codes = rng.integers(0, 16, (M, K)).astype(np.uint8)
    places = rng.permutation(K)[:2 * max(1, K // 128)].reshape(-1, 2)
    for a, b in places:
        x[:, a] = x[:, b] = 448.0
        codes[:, a] = rng.integers(4, 8, M)  # 2, 3, 4 or 6
        codes[:, b] = codes[:, a] + 8
    xt = torch.from_numpy(x).to(E4M3)
    assert np.array_equal(xt.double().numpy(), x)
    scales = np.full((M, -(-K // 32)), 127, np.uint8)
    assert 6 * K + 448 * 6 * 2 * len(places) < 2 ** 18
    w = ssm.Q4Weight.pack(torch.from_numpy(codes), torch.from_numpy(scales))
    return (xt.to(DEV), ssm.Q4Weight(w.codes.to(DEV), w.scales.to(DEV), M, K), x @ O.dequantize(codes, scales).T)


@pytest.mark.parametrize("T,M,K", [(1, 300, 1040), (3, 9000, 528), (4, 40, 4112), (7, 40, 528), (16, 300, 1040), (20, 300, 2064), (32, 130, 272),
                                   (32, 20000, 656), (40, 200, 528), (64, 384, 1040), (64, 32790, 400), (130, 257, 656), (300, 1000, 2064),
                                   (600, 3900, 1040), (1000, 4001, 272), (1510, 4090, 272), (2050, 2100, 1040), (3000, 3100, 528)])
def test_sums_of_8_bit_tokens_keep_what_outliers_leave(T, M, K):
    x, w, want = outliers(T, M, K)
    one = torch.ones(T, device=DEV)
    got = ssm.q4_linear(x, w, x_scale=one, out_dtype=torch.float32).cpu()
    exact = torch.from_numpy(want).float()
    assert torch.equal(exact.double(), torch.from_numpy(want)) and torch.equal(got, exact)
    assert torch.equal(ssm.q4_linear(x, w, x_scale=one).cpu(), exact.bfloat16())  # the output's type where none is asked for


@pytest.mark.parametrize("T", [3, 7, 20, 40, 130])
def test_a_product_beside_a_much_larger_one(T):
    """Eight neighbouring columns, one product of 1536 that another column cancels: what is left is the small one, down to 2^-20 of
    the large one."""
    K = 128
    c = torch.zeros(8, K, dtype=torch.uint8)
    c[:, 0], c[:, 3] = 7, 1      # 6 and 0.5
    c[:, 40] = 15                # -6
    w = ssm.Q4Weight.pack(c, torch.full((8, 4), 127, dtype=torch.uint8))
    w = ssm.Q4Weight(w.codes.to(DEV), w.scales.to(DEV), 8, K)
    x, one = torch.zeros(T, K, device=DEV), torch.ones(T, device=DEV)
    x[:, 0] = x[:, 40] = 256
    for e in range(8, -10, -1):
        x[:, 3] = -2.0 ** e
        for dt in (torch.float32, torch.bfloat16):
            got = ssm.q4_linear(x.to(E4M3), w, x_scale=one, out_dtype=dt).float()
            assert (got == -2.0 ** (e - 1)).all(), (e, dt, got[0, 0].item())
