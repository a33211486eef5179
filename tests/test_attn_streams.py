"""Where the attention calls take the memory of what they make, when they are given a stream.  The pool that a block comes
from belongs to a stream: a block of the current stream's pool may still be in use by work queued there, which nothing
orders before the given stream's.  Without a GPU: torch's streams and allocations are replaced."""
import contextlib

import pytest
import torch

from selective_state_space_causal_amd import attn as A


class Streams:
    def __init__(self, monkeypatch):
        self.current, self.made = "current", []
        monkeypatch.setattr(torch.cuda, "stream", self.stream)
        monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: self.current)

    @contextlib.contextmanager
    def stream(self, s):
        before, self.current = self.current, s if s is not None else self.current
        yield
        self.current = before

    def allocate(self):
        t = Block(self.current)
        self.made.append(t)
        return t


class Block:
    """An allocation: its pool's stream, and the streams that its later free waits for."""

    def __init__(self, pool):
        self.pool, self.recorded = pool, []

    def record_stream(self, s):
        self.recorded.append(s)

    def data_ptr(self):
        return 0x1000


class Like:
    device = "cuda:0"

    def __init__(self, streams):
        self.streams = streams

    def new_empty(self, shape):
        return self.streams.allocate()


@pytest.fixture
def streams(monkeypatch):
    return Streams(monkeypatch)


def test_outputs_come_from_the_given_stream_s_pool(streams):
    t, view = A._new(Like(streams), (3, 2, 8), "given")
    assert t.pool == "given" and t.recorded == ["current"]  # handed back to code on the current stream
    assert view == (0x1000, 16, 8) and streams.current == "current"


def test_outputs_without_a_stream(streams):
    t, _ = A._new(Like(streams), (3, 2, 8), None)
    assert t.pool == "current" and t.recorded == []


@pytest.fixture
def calls(streams, monkeypatch):
    """kv_read and attn_decode_step up to their entry points, on tensors without storage."""
    monkeypatch.setattr(torch, "empty", lambda *a, **k: streams.allocate())
    monkeypatch.setattr(A, "_index", lambda *a: 0)
    monkeypatch.setattr(A, "_view", lambda *a: (0, 0, 0))
    monkeypatch.setattr(A, "stream_handle", lambda s, d: 0)
    monkeypatch.setattr(A, "_decode_workspace", lambda *a: 64)

    class Entry:
        @staticmethod
        def kv_read(*a):
            return 0

        @staticmethod
        def attn_decode_step(*a):
            return 0
    monkeypatch.setattr(A, "_entry", lambda: Entry)

    class Cache:
        address, device, io_only, kv_heads, head_dim = 0, "cuda:0", None, 1, 8
        check_io = staticmethod(lambda dtype: None)
        _sizes = staticmethod(lambda: ())
    return Cache


def test_rows_read_back_come_from_the_given_stream_s_pool(streams, calls):
    k, v = A.kv_read(calls, torch.zeros(3, dtype=torch.int64), dtype=torch.float32, stream="given")
    assert [k, v] == streams.made
    for t in (k, v):
        assert t.pool == "given" and t.recorded == ["current"]


def test_workspace_comes_from_the_given_stream_s_pool(streams, calls):
    q, table = torch.zeros(1, 1, 8), torch.zeros(1, 2, dtype=torch.int32)
    out = A.attn_decode_step(q, calls, table, torch.zeros(1, dtype=torch.int32), out=torch.zeros(1, 1, 8), stream="given")
    assert out.shape == (1, 1, 8)
    (ws,) = streams.made
    assert ws.pool == "given"  # used on that stream alone: nothing to wait for


def test_rows_are_read_back_in_the_given_output_s_type(streams, calls):
    """Of either output: v_out alone as well as k_out alone."""
    f32 = torch.zeros(3, 1, 8)
    for given in (dict(k_out=f32), dict(v_out=f32)):
        types = []
        with pytest.MonkeyPatch.context() as m:
            m.setattr(A, "_view", lambda t, name, shape, dtype, device: (types.append(dtype), (0, 0, 0))[1])
            m.setattr(torch, "empty", lambda shape, dtype, device: (types.append(dtype), streams.allocate())[1])
            A.kv_read(calls, torch.zeros(3, dtype=torch.int64), stream="given", **given)
        assert types == [torch.float32] * 2, given
