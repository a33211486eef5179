"""C ABI of the residual norm and the 4-bit projections (include/ssm_block.h) without a GPU: exports and host-side
validation.  Every call below is invalid on purpose (or has no tokens) and must be answered before any HIP call, so the fake
device addresses are never dereferenced or launched on."""
import contextlib
import ctypes
import math
import os
import re

import pytest
import torch

from selective_state_space_causal_amd import _lib as L
from selective_state_space_causal_amd import block as B

pytestmark = pytest.mark.skipif(torch.cuda.device_count() > 0, reason="fake-pointer tests run only without a GPU")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "ssm_block.h")
OK, NULL, SHAPE, DTYPE, ALIGN, ALIAS, WORKSPACE = range(7)
F32, BF16, E4M3 = L.SSM_F32, L.SSM_BF16, B.SSM_E4M3
BASE, STEP = 0x7F0000000000, 1 << 36
T, D, M, K = 10, 64, 96, 208


def at(i, off=0):
    return BASE + i * STEP + off


def rows(i, width=D, off=0, stride=None):
    return B._Rows(at(i, off), width if stride is None else stride)


def pick(x, d):
    return d if x == "" else x


def test_exports_every_declared_symbol():
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(ssm_[a-z0-9_]+)\s*\(", src)))
    assert names == ["ssm_q4_codes_bytes", "ssm_q4_dequantize", "ssm_q4_linear", "ssm_q4_quantize",
                     "ssm_q4_scales_bytes", "ssm_rms_norm"]
    lib = L.load()
    for n in names:
        assert hasattr(lib, n), n


def test_a_library_without_these_entry_points_is_named():
    class Old:
        pass
    with pytest.raises(ImportError, match="earlier build"):
        B.declare(Old())


def norm(tokens=T, width=D, io=BF16, rio=BF16, oio=BF16, eps=1e-5, x="", w="", r="", ro="", o="", s=None):
    return L.load().ssm_rms_norm(tokens, width, io, rio, oio, eps, pick(x, rows(0)), pick(w, at(1)), pick(r, rows(2)),
                                 pick(ro, rows(3)), pick(o, rows(4)), s, None)


def test_norm_validation():
    assert norm(tokens=0) == OK and norm(tokens=0, x=None, w=None, r=None, ro=None, o=None) == OK
    assert norm(tokens=-1) == SHAPE and norm(tokens=2 ** 31) == SHAPE
    for width in (0, 4, 12, 32776):
        assert norm(width=width) == SHAPE
    for eps in (0.0, -1e-5, math.nan, math.inf):
        assert norm(eps=eps) == SHAPE
    assert norm(io=E4M3) == DTYPE and norm(io=3) == DTYPE and norm(oio=F32) == DTYPE and norm(io=F32, rio=BF16, oio=F32) == DTYPE
    assert norm(rio=E4M3) == DTYPE and norm(rio=7) == DTYPE
    assert norm(x=None) == NULL and norm(w=None) == NULL and norm(o=None) == NULL and norm(x=B._Rows(None, D)) == NULL
    assert norm(r=None) == NULL and norm(ro=None) == NULL
    assert norm(oio=E4M3) == NULL and norm(s=at(5)) == NULL  # 8 bits and scales go together
    assert norm(x=rows(0, off=8)) == ALIGN and norm(x=rows(0, stride=D + 4)) == ALIGN and norm(w=at(1, 8)) == ALIGN
    assert norm(r=rows(2, off=2)) == ALIGN and norm(ro=rows(3, off=4)) == ALIGN and norm(o=rows(4, off=8)) == ALIGN
    assert norm(oio=E4M3, o=rows(4, off=4), s=at(5)) == ALIGN and norm(oio=E4M3, s=at(5, 2)) == ALIGN
    assert norm(x=rows(0, stride=-D)) == SHAPE and norm(x=rows(0, stride=2 ** 22 + 8)) == SHAPE
    assert norm(o=rows(4, stride=D - 8)) == ALIAS and norm(ro=rows(3, stride=0)) == ALIAS  # rows that fall on each other
    assert norm(o=rows(0, off=D * 2)) == ALIAS               # shifted by a row: overlaps x, not in place
    assert norm(ro=rows(2, off=D * 2)) == ALIAS              # the same of the residual
    assert norm(o=rows(2)) == ALIAS and norm(o=rows(3)) == ALIAS and norm(ro=rows(0)) == ALIAS
    assert norm(oio=E4M3, o=B._Rows(at(0), 2 * D), s=at(5)) == ALIAS  # 8-bit rows over x
    assert norm(o=B._Rows(at(1), D)) == ALIAS                # over the weight
    for other in (0, 1, 2, 3, 4):
        assert norm(oio=E4M3, s=at(other)) == ALIAS, other


def q4(codes=None, scales=None, m=M, k=K):
    return B._Q4(at(10) if codes is None else codes, at(11) if scales is None else scales, m, k)


def test_norm_eps_is_a_normal_number():
    """The reciprocal root of a row of zeros and a subnormal eps would be an infinity, the row NaN."""
    for eps in (2.0 ** -149, 2.0 ** -127):
        assert norm(eps=eps) == SHAPE
    assert norm(eps=2.0 ** -126, tokens=0) == OK


def test_sizes():
    lib = L.load()
    assert lib.ssm_q4_codes_bytes(M, K) == 6 * 2 * 1024 and lib.ssm_q4_scales_bytes(M, K) == 6 * 256
    assert lib.ssm_q4_codes_bytes(1, 16) == 1024 and lib.ssm_q4_scales_bytes(17, 528) == 4 * 256
    for m, k in ((0, 16), (1, 0), (1, 8), (1, 24), (2 ** 20 + 1, 16), (1, 2 ** 20 + 16), (2 ** 20, 2 ** 19)):
        assert lib.ssm_q4_codes_bytes(m, k) == 0 and lib.ssm_q4_scales_bytes(m, k) == 0
    assert lib.ssm_q4_codes_bytes(2 ** 20, 2 ** 18) == 2 ** 37


@pytest.mark.parametrize("fn", ["quantize", "dequantize"])
def test_quantize_validation(fn):
    lib = L.load()

    def call(io=BF16, w="", q=""):
        w, q = pick(w, rows(0, K)), pick(q, q4())
        return lib.ssm_q4_quantize(io, w, q, None) if fn == "quantize" else lib.ssm_q4_dequantize(io, q, w, None)
    assert call(io=E4M3) == DTYPE
    assert call(w=None) == NULL and call(q=None) == NULL and call(q=B._Q4(None, at(11), M, K)) == NULL
    assert call(q=B._Q4(at(10), None, M, K)) == NULL and call(w=B._Rows(None, K)) == NULL
    for m, k in ((0, K), (-1, K), (2 ** 20 + 1, K), (M, 0), (M, 24), (M, 2 ** 20 + 16)):
        assert call(q=q4(m=m, k=k)) == SHAPE
    assert call(w=rows(0, stride=2 ** 22 + 8)) == SHAPE and call(w=rows(0, stride=-K)) == SHAPE
    assert call(w=rows(0, K, off=8)) == ALIGN and call(w=rows(0, stride=K + 4)) == ALIGN
    assert call(q=q4(codes=at(10, 8))) == ALIGN and call(q=q4(scales=at(11, 8))) == ALIGN
    assert call(w=rows(10, K)) == ALIAS and call(w=rows(11, K)) == ALIAS
    if fn == "quantize":
        assert call(q=q4(scales=at(10, 1024))) == ALIAS
    else:
        assert call(w=rows(0, stride=K - 8)) == ALIAS


def linear(tokens=T, x_dtype=BF16, o_dtype=BF16, x="", xs=None, q="", o=""):
    return L.load().ssm_q4_linear(tokens, x_dtype, o_dtype, pick(x, rows(0, K)), xs, pick(q, q4()), pick(o, rows(1, M)), None)


def test_linear_validation():
    assert linear(tokens=0) == OK
    assert linear(tokens=-1) == SHAPE and linear(tokens=2 ** 24) == SHAPE
    assert linear(tokens=2 ** 20, q=q4(m=2 ** 17)) == SHAPE  # more than 2^36 outputs
    assert linear(x_dtype=3) == DTYPE and linear(o_dtype=E4M3) == DTYPE
    assert linear(q=None) == NULL and linear(q=q4(k=24)) == SHAPE and linear(q=q4(m=0)) == SHAPE
    assert linear(x=None) == NULL and linear(o=None) == NULL
    assert linear(x_dtype=E4M3) == NULL and linear(xs=at(2)) == NULL  # 8 bits and scales go together
    assert linear(x=rows(0, K, off=8)) == ALIGN and linear(x=rows(0, stride=K + 4)) == ALIGN
    assert linear(o=rows(1, M, off=1)) == ALIGN and linear(o_dtype=F32, o=rows(1, M, off=2)) == ALIGN
    assert linear(x_dtype=E4M3, xs=at(2, 2)) == ALIGN and linear(q=q4(codes=at(10, 4))) == ALIGN
    assert linear(x=rows(0, stride=-16)) == SHAPE and linear(o=rows(1, stride=2 ** 22 + 1)) == SHAPE
    assert linear(o=rows(0, M)) == ALIAS and linear(o=rows(10, M)) == ALIAS and linear(o=rows(11, M)) == ALIAS
    assert linear(o=rows(1, stride=M - 1)) == ALIAS
    assert linear(x_dtype=E4M3, xs=at(2), o=rows(2, M)) == ALIAS

def test_linear_has_a_most_of_outputs():
    """What one launch's work-items can reach: 2^35 outputs."""
    lib, m = L.load(), 1 << 20
    q = B._Q4(at(2), at(6), m, K)
    for tokens, st in ((1 << 15) + 1, SHAPE), ((1 << 24) - 1, SHAPE), (1 << 15, NULL):
        assert lib.ssm_q4_linear(tokens, BF16, BF16, None, None, q, rows(5, m), None) == st



def test_python_refusals_name_the_argument():
    """Host tensors: everything is refused before a launch."""
    x, w = torch.zeros(3, 64), torch.ones(64)
    bf = torch.bfloat16
    for what, call in (
            ("tokens, width", lambda: B.rms_norm(x[0], w)), ("a GPU", lambda: B.rms_norm(x, w)),
            ("residual_out without", lambda: B.rms_norm(x, w, residual_out=x)),
            ("scale is for", lambda: B.rms_norm(x, w, scale=w)),
            ("tokens, width", lambda: B.q4_quantize(x[0])), ("multiple of 16", lambda: B.q4_quantize(x[:, :24])),
            ("a GPU", lambda: B.q4_quantize(x)), ("a GPU", lambda: B.q4_dequantize(B.Q4Weight.allocate(3, 64, "cpu"))),
            ("a GPU", lambda: B.q4_linear(x, B.Q4Weight.allocate(3, 64, "cpu"))),
            ("tokens, width", lambda: B.q4_linear(x[0], B.Q4Weight.allocate(3, 64, "cpu")))):
        with pytest.raises(ValueError, match=what):
            call()
    for call in (lambda: B.rms_norm(x.half(), w), lambda: B.rms_norm(x, w, out_dtype=bf), lambda: B.q4_quantize(x.half()),
                 lambda: B.q4_dequantize(B.Q4Weight.allocate(3, 64, "cpu"), dtype=torch.float16),
                 lambda: B.q4_linear(x.half(), B.Q4Weight.allocate(3, 64, "cpu")),
                 lambda: B.q4_linear(x, B.Q4Weight.allocate(3, 64, "cpu"), out_dtype=torch.float16)):
        with pytest.raises(TypeError):
            call()


class Streams:
    """torch's streams, devices and allocations replaced, and the entry points: what a call does up to its launch."""

    def __init__(self, monkeypatch):
        self.stream, self.device, self.made, self.launched = "current", "cuda:0", [], []
        monkeypatch.setattr(torch.cuda, "stream", lambda s: self.set("stream", s))
        monkeypatch.setattr(torch.cuda, "device", lambda d: self.set("device", d))
        monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: self.stream)
        monkeypatch.setattr(torch, "empty", self.empty)
        monkeypatch.setattr(B, "_rows", lambda *a: None)
        monkeypatch.setattr(B, "_vector", lambda *a: None)
        monkeypatch.setattr(B, "_q4", lambda *a: None)
        monkeypatch.setattr(B, "stream_handle", lambda s, d: s)
        monkeypatch.setattr(B, "_native", B._NoNative)
        monkeypatch.setattr(L, "load", lambda: self)

    @contextlib.contextmanager
    def set(self, name, value):
        before = getattr(self, name)
        setattr(self, name, value)
        yield
        setattr(self, name, before)

    def empty(self, shape, dtype, device):
        self.made.append(Block(self.stream, shape, dtype))
        return self.made[-1]

    def __getattr__(self, name):
        if not name.startswith("ssm_"):
            raise AttributeError(name)

        def entry(*args):
            self.launched.append((name, self.device, args[-1]))
            return 0
        return entry


class Block:
    """An allocation: its pool's stream, and the streams that its later free waits for."""

    def __init__(self, pool, shape, dtype):
        self.pool, self.recorded, self.shape, self.dtype = pool, [], shape, dtype

    def record_stream(self, s):
        self.recorded.append(s)


class Tensor:
    """A tensor on a second GPU, without storage."""
    device = "cuda:1"

    def __init__(self, *shape, dtype=torch.float32):
        self.shape, self.dtype = torch.Size(shape), dtype

    def dim(self):
        return len(self.shape)


@pytest.mark.parametrize("stream", [None, "given"])
def test_memory_and_launch_belong_to_the_given_stream_and_the_tensors_device(monkeypatch, stream):
    """What a call makes comes from the pool of the stream that writes it, and is not handed out again before the current
    stream is done with it; the launch is made with the tensors' device current."""
    s = Streams(monkeypatch)
    x, w = Tensor(3, 64), B.Q4Weight(Tensor(1, 1, 64, 16), Tensor(1, 1, 64, 4), 16, 64)
    B.rms_norm(x, Tensor(64), out_dtype=B.E4M3, stream=stream)
    B.q4_linear(x, w, stream=stream)
    B.q4_quantize(x, stream=stream)
    B.q4_dequantize(w, stream=stream)
    assert [n for n, _, _ in s.launched] == ["ssm_rms_norm", "ssm_q4_linear", "ssm_q4_quantize", "ssm_q4_dequantize"]
    assert all(device == "cuda:1" and at == stream for _, device, at in s.launched) and s.device == "cuda:0"
    assert [tuple(t.shape) for t in s.made] == [(3, 64), (3,), (3, 16), (1, 1, 64, 16), (1, 1, 64, 4), (16, 64)]
    for t in s.made:
        assert (t.pool, t.recorded) == (("current", []) if stream is None else ("given", ["current"]))
