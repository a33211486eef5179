"""What attn_layer.py refuses or answers without a GPU: the operators are replaced, so that nothing is launched."""
import pytest
import torch

from selective_state_space_causal_amd import attn, attn_layer


class Cache:
    kv_heads, head_dim, page_size = 1, 8, 16


def weights(d_model=4):
    return {"qkv": torch.zeros(3 * 8, d_model), "out": torch.zeros(d_model, 8)}


@pytest.fixture
def calls(monkeypatch):
    done = []

    def kv_write(k, v, cache, slots, **kw):
        done.append("kv_write")

    def kv_read(cache, slots, *, dtype=None):
        done.append("kv_read")
        return torch.zeros(2, len(slots), 1, 8)

    def attn_prefill(q, k, v, cu_q, cu_k=None):
        done.append("attn_prefill")
        return torch.zeros(q.shape)

    for f in (kv_write, kv_read, attn_prefill):
        monkeypatch.setattr(attn, f.__name__, f)
    return done


@pytest.mark.parametrize("given", [dict(context_slots=torch.arange(5)), dict(cu_k=torch.tensor([0, 2], dtype=torch.int32))])
def test_context_slots_and_cu_k_go_together(calls, given):
    """One without the other would take the wrong rows as a sequence's context; refused before the cache is written."""
    cu = torch.tensor([0, 2], dtype=torch.int32)
    with pytest.raises(ValueError, match="go together"):
        attn_layer.attn_block_prefill(torch.zeros(2, 4), weights(), 1, Cache(), torch.arange(2), cu, torch.arange(2),
                                      torch.ones(4), **given)
    assert calls == []


def test_no_tokens(calls):
    """A prompt of no tokens gives [0, d_model], as the operators do."""
    out = attn_layer.attn_block_prefill(torch.zeros(0, 4), weights(), 1, Cache(), torch.arange(0),
                                        torch.tensor([0, 0], dtype=torch.int32), torch.arange(0), torch.ones(4))
    assert out.shape == (0, 4) and calls == ["kv_write", "attn_prefill"]


def test_slots_of_a_table_without_pages():
    """No pages: no slots, and no index into the table, which would lie outside it."""
    table = torch.empty(2, 0, dtype=torch.int32)
    assert attn_layer.cache_slots(table, torch.tensor([0, 1, 1]), torch.tensor([0, 5, -1]), 16).tolist() == [-1, -1, -1]


def test_slots():
    table = torch.tensor([[3, 0, -1], [1, 2, 4]], dtype=torch.int32)
    seq, pos = torch.tensor([0, 0, 1, 0, 0, 1]), torch.tensor([5, 16, 47, 33, -1, 48])
    assert attn_layer.cache_slots(table, seq, pos, 16).tolist() == [53, 0, 79, -1, -1, -1]
