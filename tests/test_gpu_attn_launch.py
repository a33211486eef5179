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


def test_a_launch_error_is_reported_and_not_tried_again(monkeypatch):
    """The entry points replaced by ones that do nothing but report a failed launch: the native binding calls them once and
    raises; nothing has been written and the library is not asked again."""
    assert A._bound() is not A._NoNative, "the native binding is not built"
    calls, names = [], ["ssm_rope", "ssm_kv_write", "ssm_kv_read", "ssm_attn_prefill", "ssm_attn_decode_step"]
    i32, i64, f32, vp, size = ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_void_p, ctypes.c_size_t
    arguments = [(i64, i32, i32, i32, i32) + (vp,) * 6, (i64, i32, vp, vp, vp, vp, vp, i32, vp, vp, vp, vp),
                 (i64, i32) + (vp,) * 5, (vp,) * 9, (i64, i32, i32, f32, vp, vp, vp, i64, vp, vp, vp, vp, size, vp)]

    def failing(name, types):
        def entry(*args):
            calls.append(name)
            return 7  # SSM_ERR_LAUNCH
        return ctypes.CFUNCTYPE(ctypes.c_int, *types)(entry)
    stubs = [failing(n, t) for n, t in zip(names, arguments)]
    ops = operators()
    before = [[t.clone() for t in wrote] for _, _, wrote in ops]
    lib, said = A._lib.load(), {}

    class Failing:
        def __getattr__(self, name):
            return stubs[names.index(name)] if name in names else getattr(lib, name)
    A._entry()  # attn.py's own half keeps the library
    with monkeypatch.context() as m:
        m.setattr(A._lib, "load", Failing)
        A._native = None
        A._bound()
    try:
        for name, call, _ in ops:
            with pytest.raises(ssm.SsmError) as e:
                call()
            said[name] = (e.value.status, str(e.value))
    finally:
        A._native = None
        A._bound()  # the library's entry points again
    assert calls == names
    for name, (status, text) in said.items():
        assert status == 7 and name in text and "SSM_ERR_LAUNCH" in text
    for (name, _, wrote), old in zip(ops, before):
        assert all(torch.equal(a, b) for a, b in zip(wrote, old)), name
    ops[0][1]()
    assert not torch.equal(ops[0][2][0], before[0][0])  # and it rotates again


def test_a_given_stream_s_outputs_are_not_the_current_stream_s_memory():
    """A block just freed on the current stream, which work queued there may still use, is not what a call on another stream
    writes to."""
    q = torch.randn(64, HQ, D, generator=torch.Generator().manual_seed(1)).bfloat16().to(DEV)
    cu = torch.tensor([0, 64], dtype=torch.int32, device=DEV)
    want = ssm.attn_prefill(q, q, q, cu)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    freed = want.clone()
    at = freed.data_ptr()
    del freed
    got = ssm.attn_prefill(q, q, q, cu, stream=s)
    assert got.data_ptr() != at
    assert torch.empty_like(got).data_ptr() == at  # it stays the current stream's
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got, want)
