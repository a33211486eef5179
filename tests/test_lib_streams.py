"""Where the scan's, the codec's, the projections' and the layer's calls take the memory of what they make, when they are given a
stream: from that stream's pool, as the attention and block calls do; what is returned is not handed out again before the current
stream is done with it.  Without a GPU: torch's streams and allocations are replaced, and the library by one that launches nothing."""
import contextlib
import ctypes

import pytest
import torch

from selective_state_space_causal_amd import _lib as L

B, D, S, N, R = 2, 16, 8, 16, 4
F32 = torch.float32


class Block(torch.Tensor):
    """An allocation: its pool's stream, and the streams that its later free waits for."""

    def record_stream(self, s):
        self.recorded.append(s)


class Library:
    """Every entry point succeeds; sizes are not 0."""

    def __getattr__(self, name):
        return lambda *a: 64 if "bytes" in name or "blocks" in name or "floats" in name else 0


@pytest.fixture
def made(monkeypatch):
    at, made = ["current"], []

    @contextlib.contextmanager
    def stream(s):
        at.append(s)
        yield
        at.pop()

    def pooled(make):
        def alloc(*shape, **kw):
            kw.pop("device", None)
            t = make(*shape, **kw).as_subclass(Block)
            t.pool, t.recorded = at[-1], []
            made.append(t)
            return t
        return alloc
    for name in ("empty", "zeros", "empty_like"):
        monkeypatch.setattr(torch, name, pooled(getattr(torch, name)))
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: at[-1])
    monkeypatch.setattr(L, "load", Library)
    monkeypatch.setattr(L, "stream_handle", lambda s, d=None: 0)
    for name in ("_check", "_check_index"):
        monkeypatch.setattr(L, name, lambda *a, **k: None)
    return made


def t(*shape, dtype=F32):
    return torch.ones(*shape, dtype=dtype)


class OnGpu(torch.Tensor):
    device = property(lambda self: torch.device("cuda:0"))
    is_cuda = property(lambda self: True)


P = {"A": t(D, N), "Dskip": t(D), "dt_bias": t(D), "conv_w": t(D, 4)}
X, X1, BC, BC1, H, C = t(B, D, S), t(B, D), t(B, S, N), t(B, N), t(B, D, N), t(B, D, 3)
SLOTS, WX = t(B, dtype=torch.int32), t(R + 2 * N, D)


def projector():
    p = L.Projector.__new__(L.Projector)
    p.lib, p.handle, p.ws, p.ws_bytes = Library(), ctypes.c_void_p(), t(4), 4
    return p


# the call, and how many of what it makes it keeps to itself
CALLS = {
    "prefill": (lambda s: L.prefill(X, X, X, BC, BC, P, stream=s), 1),
    "decode_step": (lambda s: L.decode_step(X1, X1, X1, BC1, BC1, P, H, C, stream=s), 0),
    "prefill_pool": (lambda s: L.prefill_pool(X, X, X, BC, BC, P, SLOTS, H, C, stream=s), 0),
    "decode_step_pool": (lambda s: L.decode_step_pool(X1, X1, X1, BC1, BC1, P, SLOTS, H, C, stream=s), 0),
    "q8_quantize": (lambda s: L.q8_quantize(t(256).as_subclass(OnGpu), stream=s), 0),
    "q8_dequant_sum": (lambda s: L.q8_dequant_sum([t(256, dtype=torch.int8)], [t(2)], stream=s), 0),
    "Projector": (lambda s: projector()(L.PROJ_X, X, t(R, D), stream=s), 0),
    "conv_silu": (lambda s: L.conv_silu(X, P, stream=s), 0),
    "conv_xproj": (lambda s: L.conv_xproj(X, P, WX, R, stream=s), 0),
    "decode_fused": (lambda s: L.decode_fused(X1, X1, P, WX, t(D, R), R, H, C, stream=s), 1),
    "decode_fused_noalloc": (lambda s: L.decode_fused_noalloc(X1, X1, P, WX, t(D, R), R, H, C, stream=s), 0),
    "calib_issue": (lambda s: L.calib_issue(0, 1, 1, stream=s), 0),
    "calib_read": (lambda s: L.calib_read(t(64).as_subclass(OnGpu), stream=s), 0),
}


@pytest.mark.parametrize("stream", [None, "given"])
@pytest.mark.parametrize("name", sorted(CALLS))
def test_memory_belongs_to_the_given_stream(made, name, stream):
    call, kept = CALLS[name]
    call(stream)
    assert made
    for m in made:
        assert m.pool == (stream or "current"), tuple(m.shape)
    assert sum(m.recorded == [] for m in made) == (len(made) if stream is None else kept)
    assert all(m.recorded in ([], ["current"]) for m in made)
