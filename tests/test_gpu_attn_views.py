"""Packed projections whose heads lie in turn, used in place, against the same rows laid out apart."""
import pytest
import torch

import selective_state_space_causal_amd as ssm

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("T", [1, 33])
def test_heads_in_turn_in_place(T):
    H, D = 4, 64
    x = torch.randn(T, H, 3, D, generator=torch.Generator().manual_seed(T)).bfloat16().to(DEV)
    q, k, v = (x[:, :, i] for i in range(3))
    pos, cu = torch.arange(T, device=DEV) * 7, torch.tensor([0, T], dtype=torch.int32, device=DEV)
    freq, _ = ssm.rope_frequencies(D, device=DEV)
    kept = v.clone()
    wq, wk = ssm.rope(q.contiguous(), k.contiguous(), pos, freq)
    out = ssm.attn_prefill(wq, wk, v.contiguous(), cu)
    assert ssm.rope(q, k, pos, freq, q_out=q, k_out=k)[0] is q
    assert torch.equal(q, wq) and torch.equal(k, wk) and torch.equal(v, kept)
    assert torch.equal(ssm.attn_prefill(q, k, v, cu), out)


@pytest.mark.parametrize("T", [1, 33])
def test_groups_in_turn_written_and_rotated_in_place(T):
    H, G, D = 3, 2, 64
    x = torch.randn(T, H, G + 2, D, generator=torch.Generator().manual_seed(T)).bfloat16().to(DEV)
    before = x.clone()
    k, v = x[:, :, G], x[:, :, G + 1]
    pos = torch.arange(T, device=DEV) + 5
    freq, _ = ssm.rope_frequencies(D, device=DEV)
    want = ssm.rope(k.contiguous(), None, pos, freq)[0]
    c = ssm.KVCache.allocate(3, 16, H, D, torch.bfloat16, DEV)
    ssm.kv_write(k, v, c, torch.arange(T, device=DEV), positions=pos, freq=freq, k_out=k)
    assert torch.equal(k, want)
    for i in (0, 1, 3):
        assert torch.equal(x[:, :, i], before[:, :, i])
    ck, cv = ssm.kv_read(c, torch.arange(T, device=DEV))
    assert torch.equal(ck, want) and torch.equal(cv, before[:, :, G + 1])


def test_a_block_of_no_tokens():
    """attn_block_prefill of an empty batch of prompts."""
    from selective_state_space_causal_amd import attn_layer
    H, D, d_model = 2, 64, 128
    w = {"qkv": torch.zeros(3 * H * D, d_model, dtype=torch.bfloat16, device=DEV), "out": torch.zeros(d_model, H * D, dtype=torch.bfloat16, device=DEV)}
    c = ssm.KVCache.allocate(2, 16, H, D, torch.int8, DEV)
    none = torch.empty(0, dtype=torch.int64, device=DEV)
    out = attn_layer.attn_block_prefill(torch.empty(0, d_model, dtype=torch.bfloat16, device=DEV), w, H, c, none,
                                        torch.tensor([0, 0], dtype=torch.int32, device=DEV), none, ssm.rope_frequencies(D, device=DEV)[0])
    assert out.shape == (0, d_model)
