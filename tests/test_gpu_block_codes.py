"""The 8-bit norm's codes are the definition's, value by value, beside the borders between codes (rows up to 8192 values)."""
import pytest
import torch

import selective_state_space_causal_amd as ssm
from tests.test_block_codes import beside_borders

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("T,D", [(64, 64), (33, 264), (200, 1024), (2500, 1544), (40, 4096), (17, 8192)])
@pytest.mark.parametrize("power", [0, -20, 30])
def test_codes_beside_borders(T, D, power):
    x, want = beside_borders(T, D, seed=D)
    w = torch.full((D,), 2.0 ** -power, device=DEV)  # exact, and changes the norm's scale, not the codes
    codes, _ = ssm.rms_norm(torch.from_numpy(x).to(DEV) * 2.0 ** power, w, out_dtype=torch.float8_e4m3fn, eps=1e-20)
    got = codes.cpu().double().numpy()
    assert (got != want).sum() == 0
