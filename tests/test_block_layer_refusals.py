"""What layer.py and attn_layer.py refuse of a residual stream and of weights in 4 bits, without a GPU: the operators are
replaced, so that nothing is launched."""
import pytest
import torch

from selective_state_space_causal_amd import attn_layer, layer

B, DM, D, R, N = 2, 32, 16, 4, 16


def mixer_weights():
    return {"in_x": torch.zeros(D, DM), "in_z": torch.zeros(D, DM), "x_dt": torch.zeros(R, D), "out": torch.zeros(DM, D),
            "x_all": torch.zeros(R + 2 * N, D)}


@pytest.fixture
def launched(monkeypatch):
    """Names of the calls that would have launched something."""
    done = []

    def block_input(*args, **kw):
        done.append("block_input")
        return torch.zeros(B, DM), None

    for module in (layer, attn_layer):
        monkeypatch.setattr(module, "block_input", block_input)
    return done


@pytest.mark.parametrize("made,tokens_8bit", [(dict(), False), (dict(), True), (dict(normed=True), True),
                                              (dict(normed=True, tokens_8bit=True), False)])
def test_decode_buffers_of_another_kind(launched, made, tokens_8bit):
    """Buffers made for other tokens than the call asks for would decide in its place."""
    hidden, w = torch.zeros(B, DM), mixer_weights()
    bufs = layer.alloc_decode_buffers(hidden, w, N, True, **made)
    with pytest.raises(ValueError, match="bufs were not made with"):
        layer.mixer_decode_step(hidden, w, {"A": torch.zeros(D, N)}, None, None, None, bufs=bufs, norm=torch.ones(DM),
                                tokens_8bit=tokens_8bit)
    assert launched == []


def prefill(hidden, residual):
    w = mixer_weights()
    bufs = layer.alloc_buffers(hidden, w, N, normed=True)
    for name, call in layer.stages(hidden, w, {}, None, bufs, norm=torch.ones(DM), residual=residual):
        if name == "norm":
            return call()


def test_prompt_s_residual_has_hidden_s_shape(launched):
    """As many values in another order of rows are another stream."""
    with pytest.raises(ValueError, match="residual: shape"):
        prefill(torch.zeros(2, 5, DM), torch.zeros(5, 2, DM))
    assert launched == []


@pytest.mark.parametrize("which", ["hidden", "residual"])
def test_prompt_in_rows_that_no_one_stride_reaches(launched, which):
    """Refused: a copy of hidden would be made on another stream than the call's, one of residual would be updated in its place."""
    t = {"hidden": torch.zeros(2, 5, DM), "residual": torch.zeros(2, 5, DM)}
    t[which] = torch.zeros(5, 2, DM).transpose(0, 1)
    with pytest.raises(RuntimeError, match="view"):
        prefill(t["hidden"], t["residual"])
    assert launched == []


class Cache:
    kv_heads, head_dim, page_size = 1, 8, 16


@pytest.mark.parametrize("rows,tokens_8bit,match", [(3 * 8 + 1, False, "qkv weight"), (3 * 8, True, "4 bits")])
@pytest.mark.parametrize("decode", [False, True])
def test_attention_refuses_before_the_residual_stream_is_updated(launched, decode, rows, tokens_8bit, match):
    """A call that is put right and made again must not add hidden twice."""
    weights = {"qkv": torch.zeros(rows, DM), "out": torch.zeros(DM, 8)}
    kw = dict(norm=torch.ones(DM), residual=torch.zeros(B, DM), tokens_8bit=tokens_8bit)
    hidden, i32 = torch.zeros(B, DM), torch.int32
    with pytest.raises(ValueError, match=match):
        if decode:
            attn_layer.attn_block_decode(hidden, weights, 1, Cache(), torch.zeros(B, 1, dtype=i32), torch.ones(B, dtype=i32),
                                         torch.ones(4), **kw)
        else:
            attn_layer.attn_block_prefill(hidden, weights, 1, Cache(), torch.arange(B), torch.tensor([0, B], dtype=i32),
                                          torch.arange(B), torch.ones(4), **kw)
    assert launched == []
