"""What the attention calls make of launch errors: one left behind by an earlier, unrelated call is not theirs, and one of
their own is reported and not tried again."""
import ctypes

import pytest
import torch

import selective_state_space_causal_amd as ssm
from selective_state_space_causal_amd import attn as A

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
T, HQ, HKV, D, PAGE = 20, 4, 2, 64, 16


def hip():
    """The HIP runtime that this process uses."""
    A._bound()
    with open("/proc/self/maps") as f:
        path = next(line.split()[-1] for line in f if "libamdhip64.so" in line)
    return ctypes.CDLL(path)


def operators():
    """(name, call, tensors that the call writes) of the five operators, in place where they may be."""
    x = torch.randn(T, HQ + 2 * HKV, D, generator=torch.Generator().manual_seed(0)).bfloat16().to(DEV)
    q, k, v = x[:, :HQ], x[:, HQ:HQ + HKV], x[:, HQ + HKV:]
    c = ssm.KVCache.allocate(320, PAGE, HKV, D, torch.int8, DEV)
    for t in (c.k, c.v, c.k_scale, c.v_scale):
        t.zero_()
    pos, slots = torch.arange(T, device=DEV), torch.arange(T, device=DEV)
    freq, _ = ssm.rope_frequencies(D, device=DEV)
    ko, vo = (torch.zeros(T, HKV, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    out = torch.zeros(T, HQ, D, dtype=torch.bfloat16, device=DEV)
    cu = torch.tensor([0, T], dtype=torch.int32, device=DEV)
    table = torch.arange(320, dtype=torch.int32, device=DEV)[None]  # 5120 tokens: two launches
    n = torch.tensor([T], dtype=torch.int32, device=DEV)
    return [
        ("ssm_rope", lambda: ssm.rope(q, k, pos, freq, q_out=q, k_out=k), [x]),
        ("ssm_kv_write", lambda: ssm.kv_write(k, v, c, slots, q=q, positions=pos, freq=freq, q_out=q, k_out=k),
         [x, c.k, c.v, c.k_scale, c.v_scale]),
        ("ssm_kv_read", lambda: ssm.kv_read(c, slots, dtype=torch.bfloat16, k_out=ko, v_out=vo), [ko, vo]),
        ("ssm_attn_prefill", lambda: ssm.attn_prefill(q, k, v, cu, out=out), [out]),
        ("ssm_attn_decode_step", lambda: ssm.attn_decode_step(q[:1], c, table, n, out=out[:1]), [out]),
    ]


@pytest.mark.parametrize("native", [True, False])
def test_an_error_left_behind_is_not_the_call_s(native, monkeypatch):
    lib = hip()
    runs = [operators(), operators()]
    if not native:
        monkeypatch.setattr(A, "_native", A._NoNative)
    for (name, call, wrote), (_, plain, want) in zip(*runs):
        plain()
        assert lib.hipSetDevice(10 ** 6) != 0 and lib.hipPeekAtLastError() != 0  # refused: no such device
        call()
        for a, b in zip(wrote, want):
            same = torch.equal(a, b)
            assert same, f"{name}: not the result of one call"
