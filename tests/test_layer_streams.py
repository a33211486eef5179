"""Where a mixer layer takes the memory of what it makes, when it is given a stream: as for the attention and block calls, from the
pool of that stream, whose work writes it; nothing orders the work that is queued on the current stream before it.  Without a GPU:
torch's streams and allocations are replaced, and so are the layer's stages."""
import contextlib

import pytest
import torch

from selective_state_space_causal_amd import block, layer

B, L, DM, D, R, N = 2, 8, 32, 16, 4, 16


class Block(torch.Tensor):
    """An allocation: its pool's stream, and the streams that its later free waits for."""

    def record_stream(self, s):
        self.recorded.append(s)


class Streams:
    def __init__(self, monkeypatch):
        self.current, self.made, self.ran, empty = "current", [], [], torch.empty

        def make(*shape, **kw):
            t = empty(*shape, **kw).as_subclass(Block)
            t.pool, t.recorded = self.current, []
            self.made.append(t)
            return t
        monkeypatch.setattr(torch, "empty", make)
        monkeypatch.setattr(torch, "empty_like", lambda t: make(t.shape, dtype=t.dtype, device=t.device))
        monkeypatch.setattr(torch.cuda, "stream", self.stream)
        monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: self.current)
        for name in ("stages", "decode_stages"):
            monkeypatch.setattr(layer, name, lambda *a, **k: [("all", lambda: self.ran.append(self.current))])

    @contextlib.contextmanager
    def stream(self, s):
        before, self.current = self.current, s if s is not None else self.current
        yield
        self.current = before


@pytest.mark.parametrize("four_bit", [False, True])
@pytest.mark.parametrize("stream", [None, "given"])
@pytest.mark.parametrize("decode", [False, True])
def test_a_layer_s_memory_belongs_to_the_given_stream(monkeypatch, decode, stream, four_bit):
    w = {k: torch.zeros(s) for k, s in dict(in_x=(D, DM), in_z=(D, DM), out=(DM, D), x_dt=(R, D), x_all=(R + 2 * N, D)).items()}
    if four_bit:
        for k in ("in_x", "in_z", "out"):
            w[k] = block.Q4Weight.allocate(*w[k].shape, device="cpu")
    params, norm = {"A": torch.zeros(D, N)}, torch.ones(DM)
    s = Streams(monkeypatch)
    if decode:
        out = layer.mixer_decode_step(torch.zeros(B, DM), w, params, None, None, None, stream=stream, norm=norm, tokens_8bit=four_bit)
        returned = [t for t in s.made if t.shape == (B, 1, DM)]
        assert len(returned) == 1 and out.data_ptr() == returned[0].data_ptr()
    else:
        returned = layer.mixer_prefill(torch.zeros(B, L, DM), w, params, None, stream=stream, norm=norm)
        assert len(returned) == 3
    here = stream or "current"
    assert len(s.made) > 3 and s.ran == [here] and s.current == "current"  # what a stage makes is from there too
    for t in s.made:
        assert t.pool == here, tuple(t.shape)
    for t in returned:  # handed back to code on the current stream
        assert t.recorded == ([] if stream is None else ["current"]), tuple(t.shape)
