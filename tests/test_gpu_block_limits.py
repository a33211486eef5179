"""The magnitudes that the norm and the 4-bit products are documented for, at their ends."""
import pytest
import torch

import selective_state_space_causal_amd as ssm

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("D", [64, 4096, 32768])
def test_norm_of_the_largest_magnitudes(D):
    """The sum of 2^15 squares of (just below) 2^56 is below 2^127: every value is its row's root mean square."""
    x = torch.full((3, D), 2.0 ** 56 * (1 - 2.0 ** -24), device=DEV)
    x[:, ::2] *= -1
    w = torch.ones(D, device=DEV)
    # a row of one magnitude: the mean of squares is off by its additions' rounding, 2^-19 of a value as in the norm's other tests
    assert ((ssm.rms_norm(x, w) * x.sign() - 1).abs() <= 2.0 ** -19).all()
    codes, scale = ssm.rms_norm(x, w, out_dtype=torch.float8_e4m3fn)
    assert (codes.float() == 448 * x.sign()).all() and ((scale * 448 - 1).abs() <= 2.0 ** -18).all()


@pytest.mark.parametrize("T", [1, 3, 17, 40, 300])
@pytest.mark.parametrize("lo,hi", [(-99, -90), (-1, 0), (120, 127)])
def test_fp32_tokens_keep_all_their_bits(T, lo, hi):
    """Three bf16 parts of 24 bits: by the identity, every token comes back as it was."""
    K = 144
    c = torch.zeros(K, K, dtype=torch.uint8)
    c[torch.arange(K), torch.arange(K)] = 2  # 1.0
    w = ssm.Q4Weight.pack(c, torch.full((K, -(-K // 32)), 127, dtype=torch.uint8))
    w = ssm.Q4Weight(w.codes.to(DEV), w.scales.to(DEV), K, K)
    g = torch.Generator().manual_seed(T)
    e = torch.randint(lo, hi, (T, K), generator=g)
    m = torch.randint(1 << 23, 1 << 24, (T, K), generator=g)
    m[:, :8] = torch.tensor([1 << 23, (1 << 24) - 1, (1 << 23) + 1, (1 << 23) + (1 << 15), (1 << 23) + (3 << 14) + 1, (1 << 24) - (1 << 15),
                             (1 << 23) + (1 << 15) + (1 << 7), (1 << 24) - (1 << 15) - 1])
    x = (m.double() * 2.0 ** -23 * torch.exp2(e.double())).float() * torch.where(torch.rand(T, K, generator=g) < 0.5, -1.0, 1.0)
    assert torch.equal(x.abs().double(), m.double() * 2.0 ** -23 * torch.exp2(e.double()))
    assert torch.equal(ssm.q4_linear(x.to(DEV), w).cpu(), x)
