"""Sizes at which the attention kernels' 32-bit indexes would wrap, answered on the host (no GPU: the addresses are fake and
never used)."""
import pytest
import torch

from selective_state_space_causal_amd import _lib as L
from selective_state_space_causal_amd import attn as A

pytestmark = pytest.mark.skipif(torch.cuda.device_count() > 0, reason="fake-pointer tests run only without a GPU")
SHAPE, LAUNCH = 2, 7
BASE = 0x7F0000000000


def prefill(tq, tk, hq=1, hk=1):
    """One sequence of head_dim 8; k and v of token stride 0, as an expanded tensor has, take no memory to speak of."""
    d = A._Dims(1, tq, tk, hq, hk, 8, L.SSM_BF16, 1, 0.5)
    q, k, v, out = (A._View(BASE + (i << 40), s, 8) for i, s in enumerate((hq * 8, 0, 0, hq * 8)))
    return L.load().ssm_attn_prefill(d, q, k, v, BASE + (8 << 40), BASE + (9 << 40), out, None, None)


def test_keys_past_a_tile_stay_below_two_to_31():
    """Kernels step up to 256 keys past a sequence's end: from 2^31 - 256 keys on an int wraps, and the walk along the
    keys goes on from far before them."""
    for tk in (2 ** 31 - 1, 2 ** 31 - 256, 2 ** 31 - 2 ** 20):
        assert prefill(1, tk) == SHAPE, tk
    assert prefill(1, 2 ** 31 - 2 ** 20 - 1) == LAUNCH  # as far as a launch, and no device


@pytest.mark.parametrize("hq", [1, 16])
def test_rows_of_a_tile_search_stay_below_two_to_31(hq):
    """64 sequences' tiles of 32 rows are summed in an int, whatever the offsets hold."""
    most = 2 ** 30 - 32
    assert 64 * -(-most // 32) < 2 ** 31 <= 64 * -(-(most + 32) // 32)
    for tq in (most // hq + 1, (2 ** 31 - 1) // hq):
        assert prefill(tq, 1, hq) == SHAPE, tq
    assert prefill(most // hq, 1, hq) == LAUNCH
