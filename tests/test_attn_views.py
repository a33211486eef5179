"""Which views the attention calls take for an output next to an input: all that share no byte in the usual packed layouts,
and none that shares one (no GPU: the addresses are fake and never used)."""
import random

import pytest
import torch

from selective_state_space_causal_amd import _lib as L
from selective_state_space_causal_amd import attn as A

pytestmark = pytest.mark.skipif(torch.cuda.device_count() > 0, reason="fake-pointer tests run only without a GPU")
ALIAS, LAUNCH = 5, 7
BASE, FAR = 0x7F0000000000, 0x7E0000000000
D = 8


def view(at, ts, hs):
    """A view that starts `at` elements (bf16) into the buffer."""
    return A._View(BASE + 2 * at, ts, hs)


def rope(T, hq, hk, q, qo, k, ko):
    r = A._Rope(FAR, FAR + (1 << 36), D // 2, 0, 1.0)
    return L.load().ssm_rope(T, hq, hk, D, L.SSM_BF16, r, q, qo, k, ko, None)


def test_heads_side_by_side_in_place():
    """[T, 3 H, D]: q, k and v heads of a token in blocks."""
    T, H = 5, 4
    v = [view(i * H * D, 3 * H * D, D) for i in range(3)]
    assert rope(T, H, H, v[0], v[0], v[1], v[1]) == LAUNCH


def test_heads_in_turn_in_place():
    """[T, H, 3, D]: each head's q, k and v next to one another."""
    T, H = 5, 4
    v = [view(i * D, 3 * H * D, 3 * D) for i in range(3)]
    assert rope(T, H, H, v[0], v[0], v[1], v[1]) == LAUNCH
    assert rope(T, H, H, v[0], v[2], v[1], v[1]) == LAUNCH      # into the third's place
    assert rope(T, H, H, v[0], v[0], v[1], v[0]) == ALIAS
    assert rope(1, H, H, *(A._View(x.data, 0, x.head_stride) for x in (v[0], v[0], v[1], v[1]))) == LAUNCH  # one token


def test_groups_in_turn():
    """[T, Hkv, G + 2, D]: a key head's queries, key and value next to one another; the rotated keys in place."""
    T, H, G = 5, 4, 3
    k, v = (view((G + i) * D, H * (G + 2) * D, (G + 2) * D) for i in range(2))
    far = [FAR + (i << 36) for i in range(2, 8)]
    c = A._Cache(far[0], far[1], far[2], far[3], 8, 16, H, D, A.KV_I8)
    r = A._Rope(FAR, FAR + (1 << 36), D // 2, 0, 1.0)
    assert L.load().ssm_kv_write(T, L.SSM_BF16, c, far[4], k, v, r, 0, None, None, k, None) == LAUNCH
    assert L.load().ssm_kv_write(T, L.SSM_BF16, c, far[4], k, v, r, 0, None, None, v, None) == ALIAS


def elements(at, ts, hs, T, H):
    return {at + t * ts + h * hs + e for t in range(T) for h in range(H) for e in range(D)}


def test_shared_bytes_are_never_taken():
    """Strides and places at random, against the sets of elements."""
    rng = random.Random(5)
    shared = taken = 0
    for _ in range(20000):
        T, H = rng.randint(1, 4), rng.randint(1, 4)
        hs = D * rng.randint(1, 5)
        ts = rng.choice([D * rng.randint(1, 20), hs * rng.randint(1, 6), H * hs])
        same = rng.random() < 0.7
        hs2, ts2 = (hs, ts) if same else (D * rng.randint(1, 5), D * rng.randint(1, 20))
        at, at2 = D * rng.randint(0, 12), D * rng.randint(0, 12) + rng.choice([0, 0, 0, 8])
        a, b = elements(at, ts, hs, T, H), elements(at2, ts2, hs2, T, H)
        st = rope(T, H, 0, view(at, ts, hs), view(at2, ts2, hs2), None, None)
        if (at, ts, hs) != (at2, ts2, hs2) and a & b or len(b) < T * H * D:
            shared += 1
            assert st == ALIAS, (T, H, at, ts, hs, at2, ts2, hs2)
        taken += st == LAUNCH
    assert shared > 2000 and taken > 2000
