"""ctypes binding of the attention operators of include/ssm_attn.h: rotary positions, the paged
key/value cache (written quantised, read back), attention over packed prompts, and attention of one
token per sequence against the cache.  Argument marshalling only: every step runs in the library's
HIP kernels, there is no fallback.

[T, H, D] tensors may be views with any token and head strides that are multiples of 16 bytes (the
heads of a packed q/k/v projection are used in place); the D values of a head are contiguous."""
from __future__ import annotations

import ctypes
import functools
import math
import struct
import warnings
from typing import Optional

import torch

from . import _lib
from ._lib import SSM_BF16, SSM_F32, SsmError, stream_handle

KV_IO, KV_I8, KV_E4M3 = 0, 1, 2
MIN_PAGE, MAX_PAGE = 16, 1024
MAX_HEAD_DIM = 256

_IO = {torch.float32: SSM_F32, torch.bfloat16: SSM_BF16}
_CODES = {torch.int8: KV_I8, torch.float8_e4m3fn: KV_E4M3}


class _View(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64)]


class _Cache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("pages", ctypes.c_int64), ("page_size", ctypes.c_int32),
                ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("kv_dtype", ctypes.c_int32)]


class _Rope(ctypes.Structure):
    _fields_ = [("positions", ctypes.c_void_p), ("freq", ctypes.c_void_p), ("pairs", ctypes.c_int32),
                ("interleaved", ctypes.c_int32), ("mscale", ctypes.c_float)]


class _Dims(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("q_tokens", ctypes.c_int64), ("k_tokens", ctypes.c_int64),
                ("q_heads", ctypes.c_int32), ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("io_dtype", ctypes.c_int32), ("causal", ctypes.c_int32), ("scale", ctypes.c_float)]


def declare(lib):
    """Argument types of the entry points (called once by _lib.load)."""
    vp, i64, i32, pv = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.POINTER(_View)
    pc, pr = ctypes.POINTER(_Cache), ctypes.POINTER(_Rope)
    lib.ssm_rope.restype = ctypes.c_int
    lib.ssm_rope.argtypes = [i64, i32, i32, i32, i32, pr, pv, pv, pv, pv, vp]
    lib.ssm_kv_write.restype = ctypes.c_int
    lib.ssm_kv_write.argtypes = [i64, i32, pc, vp, pv, pv, pr, i32, pv, pv, pv, vp]
    lib.ssm_kv_read.restype = ctypes.c_int
    lib.ssm_kv_read.argtypes = [i64, i32, pc, vp, pv, pv, vp]
    lib.ssm_attn_prefill.restype = ctypes.c_int
    lib.ssm_attn_prefill.argtypes = [ctypes.POINTER(_Dims), pv, pv, pv, vp, vp, pv, vp, vp]
    lib.ssm_attn_decode_workspace_bytes.restype = ctypes.c_size_t
    lib.ssm_attn_decode_workspace_bytes.argtypes = [i64, i32, pc, i64]
    lib.ssm_attn_decode_step.restype = ctypes.c_int
    lib.ssm_attn_decode_step.argtypes = [i64, i32, i32, ctypes.c_float, pc, pv, vp, i64, vp, pv, vp, vp,
                                         ctypes.c_size_t, vp]


class _Calls:
    """The entry points, taking the structures above by address: a call packs its structures into one buffer of
    its own (_pack) instead of building an object for each, a third of the time a small call takes."""

    def __init__(self, lib):
        vp, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32

        def entry(name, *args):
            return ctypes.CFUNCTYPE(ctypes.c_int, *args)((name, lib))
        self.rope = entry("ssm_rope", i64, i32, i32, i32, i32, vp, vp, vp, vp, vp, vp)
        self.kv_write = entry("ssm_kv_write", i64, i32, vp, vp, vp, vp, vp, i32, vp, vp, vp, vp)
        self.kv_read = entry("ssm_kv_read", i64, i32, vp, vp, vp, vp, vp)
        self.attn_prefill = entry("ssm_attn_prefill", vp, vp, vp, vp, vp, vp, vp, vp, vp)
        self.attn_decode_step = entry("ssm_attn_decode_step", i64, i32, i32, ctypes.c_float, vp, vp, vp, i64, vp, vp, vp,
                                      vp, ctypes.c_size_t, vp)


_calls = None
_native = None  # the usual case of the calls below, natively (csrc/attn_binding.cpp); NotImplemented for any other


class _NoNative:
    """Every case goes through this file."""

    @staticmethod
    def _not_usual(*args):
        return NotImplemented
    describe = rope = kv_write = kv_read = attn_prefill = attn_decode_step = _not_usual


def _entry() -> _Calls:
    global _calls
    if _calls is None:
        _calls = _Calls(_lib.load())
    return _calls


def _bound():
    global _native
    if _native is None:
        lib = _lib.load()
        try:
            from . import _attn_fast
            _attn_fast.bind(lib.ssm_abi_version(), *(ctypes.cast(getattr(lib, n), ctypes.c_void_p).value for n in (
                "ssm_rope", "ssm_kv_write", "ssm_kv_read", "ssm_attn_prefill", "ssm_attn_decode_step",
                "ssm_attn_decode_workspace_bytes")), _fail)
            _native = _attn_fast
        except (ImportError, TypeError) as e:  # TypeError: built before versions were compared
            warnings.warn(f"the attention calls' native binding is not built for this library ({e}): small calls are slower; run "
                          "selective_state_space_causal_amd/build.py")
            _native = _NoNative
    return _native


_I32, _I64, _F32, _F64 = torch.int32, torch.int64, torch.float32, torch.float64
_VIEW = 24  # bytes of a _View
_Buffer = ctypes.c_char * 192
_two_views = struct.Struct("QqqQqq").pack_into
_views_rope = struct.Struct("QqqQqqQqqQqqQQiif4x").pack_into
_five_views_rope = struct.Struct("QqqQqqQqqQqqQqqQQiif4x").pack_into
_four_views_dims = struct.Struct("QqqQqqQqqQqqqqqiiiiif").pack_into
_cache_fields = struct.Struct("QQQQqiiii").pack_into
_no_view = (0, 0, 0)


def _io(t: torch.Tensor) -> int:
    code = _IO.get(t.dtype)
    if code is None:
        raise TypeError(f"io tensors must be float32 or bfloat16, got {t.dtype}")
    return code


def _view(t: torch.Tensor, name: str, shape, dtype, device):
    """A [T, H, D] tensor's view, checked for shape, dtype, GPU device and contiguous heads."""
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if t.device != device or not t.is_cuda:
        raise ValueError(f"{name} must be on {device} (a GPU)")
    ts, hs, one = t.stride()
    if one != 1 and shape[2] != 1:
        raise ValueError(f"{name}: the values of a head must be contiguous (stride {one})")
    # the stride of an axis of length 1 is never used, and torch leaves it arbitrary
    return t.data_ptr(), ts if shape[0] > 1 else 0, hs if shape[1] > 1 else 0


def _made(make, stream, device, returned=True):
    """make()'s tensor, from the memory pool of the stream that writes it: a block of the current stream's pool may still
    be in use by work queued there, which nothing orders before `stream`'s.  A returned one is used on the
    current stream, so its memory is not handed out again before that is done with it."""
    if stream is None:
        return make()
    with torch.cuda.stream(stream):
        t = make()
    if returned:
        t.record_stream(torch.cuda.current_stream(device))
    return t


def _new(like: torch.Tensor, shape, stream):
    """A contiguous output [T, H, D] and its view."""
    t = _made(lambda: like.new_empty(shape), stream, like.device)
    return t, (t.data_ptr(), shape[1] * shape[2], shape[2])


def _three(t, name):
    if t.dim() != 3:
        raise ValueError(f"{name} must be [tokens, heads, head_dim], got {tuple(t.shape)}")
    return t.shape


def _index(t: torch.Tensor, name: str, shape, dtype, device):
    if t.shape == shape and t.dtype == dtype and t.device == device and t.is_contiguous():
        return t.data_ptr()
    raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on {device}, got "
                     f"{t.dtype} {tuple(t.shape)} on {t.device}")


def _fail(name, st):
    raise SsmError(name, st, _lib.load().ssm_status_str(st).decode())


# ---------------------------------------------------------------- rotary positions

def rope_frequencies(rot_dim: int, *, base: float = 10000.0, scaling: Optional[str] = None, factor: float = 1.0,
                     original_max: int = 4096, beta_fast: float = 32.0, beta_slow: float = 1.0, device="cuda"):
    """(freq, mscale): the radians per position of each of the rot_dim / 2 pairs (fp64, on device),
    and the factor on cos and sin.  freq_i = base^(-2 i / rot_dim); for contexts longer than the model
    was trained on, `scaling` is
      "linear"  positions divided by factor
      "ntk"     base * factor^(rot_dim / (rot_dim - 2)): the slowest pair is slowed by factor, the
                fastest kept
      "yarn"    pairs that turn more than beta_fast times over original_max tokens are kept, those that
                turn less than beta_slow times are slowed by factor, a linear ramp between, and
                mscale = 0.1 ln(factor) + 1 for factors above 1 (Peng et al., "YaRN", 2023)."""
    if rot_dim < 2 or rot_dim % 2:
        raise ValueError(f"rot_dim must be even and at least 2, got {rot_dim}")
    if not (base > 1.0 and math.isfinite(base)) or not (factor > 0.0 and math.isfinite(factor)):
        raise ValueError("base must be above 1 and factor above 0")
    if scaling is None and factor != 1.0:
        raise ValueError(f"a factor of {factor} needs a scaling: 'linear', 'ntk' or 'yarn'")
    i = torch.arange(rot_dim // 2, dtype=torch.float64)
    mscale = 1.0
    if scaling == "ntk":
        if rot_dim < 4:
            raise ValueError("ntk scaling needs rot_dim of at least 4")
        base = base * factor ** (rot_dim / (rot_dim - 2))
    freq = torch.tensor(base, dtype=torch.float64) ** (-2.0 * i / rot_dim)
    if scaling == "linear":
        freq = freq / factor
    elif scaling == "yarn":
        def pair_of(turns):
            return rot_dim * math.log(original_max / (turns * 2 * math.pi)) / (2 * math.log(base))
        lo, hi = max(0, math.floor(pair_of(beta_fast))), min(rot_dim - 1, math.ceil(pair_of(beta_slow)))
        ramp = ((i - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
        freq = freq / factor * ramp + freq * (1 - ramp)
        mscale = 0.1 * math.log(factor) + 1.0 if factor > 1.0 else 1.0
    elif scaling not in (None, "ntk"):
        raise ValueError(f"scaling must be None, 'linear', 'ntk' or 'yarn', got {scaling!r}")
    return freq.to(device), mscale


def _rope_fields(positions, freq, interleaved, mscale, T, device):
    pairs = freq.numel()
    return (_index(positions, "positions", (T,), _I64, device), _index(freq, "freq", (pairs,), _F64, device),
            pairs, bool(interleaved), mscale)


def rope(q, k, positions, freq, *, interleaved: bool = False, mscale: float = 1.0, q_out=None, k_out=None,
         stream=None):
    """ssm_rope: q [T, Hq, D] and k [T, Hkv, D] (or None) rotated by positions [T] int64; freq (and
    mscale) as rope_frequencies gives them.  Returns (q_out, k_out); pass q_out=q, k_out=k for in place."""
    if stream is None:
        r = (_native or _bound()).rope(q, k, positions, freq, interleaved, mscale, q_out, k_out)
        if r is not NotImplemented:
            return r
    call = _entry().rope
    T, Hq, D = shape = _three(q, "q")
    dev, dtype = q.device, q.dtype
    io = _io(q)
    vq = _view(q, "q", shape, dtype, dev)
    desc = _rope_fields(positions, freq, interleaved, mscale, T, dev)
    Hk, vk, vko = 0, _no_view, _no_view
    if k is not None:
        Hk = _three(k, "k")[1]
        kshape = (T, Hk, D)
        vk = _view(k, "k", kshape, dtype, dev)
        if k_out is None:
            k_out, vko = _new(q, kshape, stream)
        else:
            vko = _view(k_out, "k_out", kshape, dtype, dev)
    elif k_out is not None:
        raise ValueError("k_out without k")
    if q_out is None:
        q_out, vqo = _new(q, shape, stream)
    else:
        vqo = _view(q_out, "q_out", shape, dtype, dev)
    buf = _Buffer()
    _views_rope(buf, 0, *vq, *vqo, *vk, *vko, *desc)
    at = ctypes.addressof(buf)
    st = call(T, Hq, Hk, D, io, at + 4 * _VIEW, at, at + _VIEW, at + 2 * _VIEW if Hk else None,
              at + 3 * _VIEW if Hk else None, stream_handle(stream, dev))
    if st != 0:
        _fail("ssm_rope", st)
    return q_out, k_out


# ---------------------------------------------------------------- the paged cache

class KVCache:
    """A paged key/value cache: k and v [pages, Hkv, page_size, D] in the io dtype, int8 or
    float8_e4m3fn, and for the 8-bit types k_scale and v_scale [pages, Hkv, page_size] fp32.  The
    tensors are the caller's; this holds them and their description."""

    __slots__ = ("k", "v", "k_scale", "v_scale", "_desc", "address", "device", "kv_heads", "head_dim", "page_size", "pages",
                 "io_only", "index", "is_bf16")

    def __init__(self, k, v, k_scale=None, v_scale=None):
        self._desc = desc = _Buffer()  # a _Cache
        self.address = at = ctypes.addressof(desc)
        r = (_native or _bound()).describe(at, k, v, k_scale, v_scale)
        if r is NotImplemented:
            r = self._describe(desc, k, v, k_scale, v_scale)
        self.pages, self.kv_heads, self.page_size, self.head_dim, self.index, self.is_bf16 = r
        self.k, self.v, self.k_scale, self.v_scale, self.device = k, v, k_scale, v_scale, k.device
        self.io_only = None if self.is_bf16 is None else k.dtype  # the io dtype that a cache of that dtype is tied to

    def _describe(self, desc, k, v, ks, vs):
        """The checks, by name; fills desc."""
        if k.dim() != 4:
            raise ValueError(f"k must be [pages, heads, page_size, head_dim], got {tuple(k.shape)}")
        shape, dtype, dev = k.shape, k.dtype, k.device
        kind = _CODES.get(dtype, KV_IO)
        if kind == KV_IO:
            if dtype not in _IO:
                raise TypeError(f"a cache holds float32, bfloat16, int8 or float8_e4m3fn, got {dtype}")
            if ks is not None or vs is not None:
                raise ValueError("k_scale and v_scale: only the 8-bit types have scales")
        else:
            self._refuse(ks, "k_scale", shape[:3], _F32, dev)
            self._refuse(vs, "v_scale", shape[:3], _F32, dev)
        self._refuse(k, "k", shape, dtype, dev)
        self._refuse(v, "v", shape, dtype, dev)
        pages, heads, page_size, dim = shape
        _cache_fields(desc, 0, k.data_ptr(), v.data_ptr(), 0 if ks is None else ks.data_ptr(), 0 if vs is None else vs.data_ptr(),
                      pages, page_size, heads, dim, kind)
        return pages, heads, page_size, dim, dev.index, None if kind != KV_IO else dtype == torch.bfloat16

    def _sizes(self):
        return self.pages, self.page_size, self.kv_heads, self.head_dim

    @staticmethod
    def _refuse(t, name, shape, dtype, dev):
        if t is None:
            raise ValueError(f"{name} is required")
        if t.shape != shape or t.dtype != dtype or t.device != dev or not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on {dev} (a GPU),"
                             f" got {t.dtype} {tuple(t.shape)} on {t.device}")

    @classmethod
    def allocate(cls, pages: int, page_size: int, kv_heads: int, head_dim: int, dtype=torch.float8_e4m3fn,
                 device="cuda"):
        """A cache with uninitialised contents (a row is written before a sequence's length covers it)."""
        k = torch.empty(pages, kv_heads, page_size, head_dim, dtype=dtype, device=device)
        scale = [torch.empty(k.shape[:3], device=device) for _ in range(2)] if dtype in _CODES else [None, None]
        return cls(k, torch.empty_like(k), *scale)

    def check_io(self, dtype):
        if self.io_only is not None and self.io_only != dtype:
            raise TypeError(f"a cache of {self.k.dtype} is written and read in that type, got {dtype}")


def kv_write(k, v, cache: KVCache, slots, *, q=None, positions=None, freq=None, interleaved: bool = False,
             mscale: float = 1.0, q_out=None, k_out=None, stream=None):
    """ssm_kv_write: keys and values k, v [T, Hkv, D] into the cache rows slots [T] int64 (page *
    page_size + place; out of range: skipped).  With positions and freq the keys are rotated on the way, and q
    [T, Hq, D] too where given; a k_out tensor receives the rotated keys.  Returns q_out (None without q)."""
    if stream is None:
        r = (_native or _bound()).kv_write(k, v, cache.address, cache.index, cache.is_bf16, slots, q, positions, freq,
                                           interleaved, mscale, q_out, k_out)
        if r is not NotImplemented:
            return r
    call = _entry().kv_write
    T = _three(k, "k")[0]
    dev, dtype = cache.device, k.dtype
    shape = (T, cache.kv_heads, cache.head_dim)
    cache.check_io(dtype)
    io = _io(k)
    vk, vv = _view(k, "k", shape, dtype, dev), _view(v, "v", shape, dtype, dev)
    ps = _index(slots, "slots", (T,), _I64, dev)
    Hq, vq, vqo, vko, desc = 0, _no_view, _no_view, _no_view, None
    if (positions is None) != (freq is None):
        raise ValueError("positions and freq go together")
    if positions is not None:
        desc = _rope_fields(positions, freq, interleaved, mscale, T, dev)
        if k_out is not None:
            vko = _view(k_out, "k_out", shape, dtype, dev)
        if q is not None:
            Hq = _three(q, "q")[1]
            qshape = (T, Hq, cache.head_dim)
            vq = _view(q, "q", qshape, dtype, dev)
            if q_out is None:
                q_out, vqo = _new(q, qshape, stream)
            else:
                vqo = _view(q_out, "q_out", qshape, dtype, dev)
    elif q is not None or k_out is not None:
        raise ValueError("q and k_out are for a call with positions and freq")
    if q is None and q_out is not None:
        raise ValueError("q_out without q")
    buf = _Buffer()
    at = ctypes.addressof(buf)
    if desc is None:
        _two_views(buf, 0, *vk, *vv)
        st = call(T, io, cache.address, ps, at, at + _VIEW, None, 0, None, None, None, stream_handle(stream, dev))
    else:
        _five_views_rope(buf, 0, *vk, *vv, *vq, *vqo, *vko, *desc)
        st = call(T, io, cache.address, ps, at, at + _VIEW, at + 5 * _VIEW, Hq, at + 2 * _VIEW if Hq else None,
                  at + 3 * _VIEW if Hq else None, at + 4 * _VIEW if k_out is not None else None,
                  stream_handle(stream, dev))
    if st != 0:
        _fail("ssm_kv_write", st)
    return q_out


def kv_read(cache: KVCache, slots, *, dtype=None, k_out=None, v_out=None, stream=None):
    """ssm_kv_read: the rows at slots [T] int64 as (k, v) [T, Hkv, D] in dtype (where not given that of
    k_out or v_out, else the cache's own, bfloat16 for the 8-bit types); slots out of range read as zeros."""
    if dtype is None:
        given = k_out if k_out is not None else v_out
        dtype = given.dtype if given is not None else cache.io_only or torch.bfloat16
    if stream is None and dtype in _IO:
        r = (_native or _bound()).kv_read(cache.address, cache.index, cache.is_bf16, slots, dtype == torch.bfloat16, k_out,
                                          v_out)
        if r is not NotImplemented:
            return r
    call = _entry().kv_read
    dev = cache.device
    if slots.dim() != 1:
        raise ValueError(f"slots must have one axis, got {tuple(slots.shape)}")
    T = slots.shape[0]
    cache.check_io(dtype)
    if dtype not in _IO:
        raise TypeError(f"io tensors must be float32 or bfloat16, got {dtype}")
    shape = (T, cache.kv_heads, cache.head_dim)
    ps = _index(slots, "slots", (T,), _I64, dev)
    views, outs = [], []
    for t, name in ((k_out, "k_out"), (v_out, "v_out")):
        if t is None:
            t = _made(lambda: torch.empty(shape, dtype=dtype, device=dev), stream, dev)
            views.append((t.data_ptr(), shape[1] * shape[2], shape[2]))
        else:
            views.append(_view(t, name, shape, dtype, dev))
        outs.append(t)
    buf = _Buffer()
    _two_views(buf, 0, *views[0], *views[1])
    at = ctypes.addressof(buf)
    st = call(T, _IO[dtype], cache.address, ps, at, at + _VIEW, stream_handle(stream, dev))
    if st != 0:
        _fail("ssm_kv_read", st)
    return outs[0], outs[1]


# ---------------------------------------------------------------- attention

def attn_prefill(q, k, v, cu_q, cu_k=None, *, causal: bool = True, scale: Optional[float] = None, out=None, lse=None,
                 stream=None):
    """ssm_attn_prefill: softmax attention of packed sequences, q [Tq, Hq, D] over k, v [Tk, Hkv, D].
    Sequence b holds rows cu_q[b] : cu_q[b + 1] of q and cu_k[b] : cu_k[b + 1] of k and v (int32 on the GPU; cu_k
    defaults to cu_q); causal lets its last query see all its keys, the one before one less, and so on.  scale
    defaults to 1 / sqrt(D).  A query that sees no key gives zeros.  Returns out [Tq, Hq, D]; an lse tensor
    [Tq, Hq] fp32 receives the log of the softmax sums."""
    if stream is None:
        r = (_native or _bound()).attn_prefill(q, k, v, cu_q, cu_q if cu_k is None else cu_k, causal, scale, out, lse)
        if r is not NotImplemented:
            return r
    call = _entry().attn_prefill
    Tq, Hq, D = shape = _three(q, "q")
    Tk, Hkv, _ = _three(k, "k")
    dev, dtype = q.device, q.dtype
    io = _io(q)
    cu_k = cu_q if cu_k is None else cu_k
    if cu_q.dim() != 1 or cu_q.shape[0] < 2:
        raise ValueError(f"cu_q must be [batch + 1] with batch >= 1, got {tuple(cu_q.shape)}")
    ends = cu_q.shape
    kshape = (Tk, Hkv, D)
    vq = _view(q, "q", shape, dtype, dev)
    vk, vv = _view(k, "k", kshape, dtype, dev), _view(v, "v", kshape, dtype, dev)
    pq, pk = _index(cu_q, "cu_q", ends, _I32, dev), _index(cu_k, "cu_k", ends, _I32, dev)
    if out is None:
        out, vo = _new(q, shape, stream)
    else:
        vo = _view(out, "out", shape, dtype, dev)
    pl = None if lse is None else _index(lse, "lse", (Tq, Hq), _F32, dev)
    buf = _Buffer()
    _four_views_dims(buf, 0, *vq, *vk, *vv, *vo, ends[0] - 1, Tq, Tk, Hq, Hkv, D, io, bool(causal),
                     D ** -0.5 if scale is None else scale)
    at = ctypes.addressof(buf)
    st = call(at + 4 * _VIEW, at, at + _VIEW, at + 2 * _VIEW, pq, pk, at + 3 * _VIEW, pl, stream_handle(stream, dev))
    if st != 0:
        _fail("ssm_attn_prefill", st)
    return out


@functools.lru_cache(maxsize=256)
def _decode_workspace(batch, q_heads, pages, page_size, kv_heads, head_dim, table_width):
    sizes = _Cache(None, None, None, None, pages, page_size, kv_heads, head_dim, KV_IO)
    return int(_lib.load().ssm_attn_decode_workspace_bytes(batch, q_heads, sizes, table_width))


def attn_decode_workspace_bytes(batch: int, q_heads: int, cache: KVCache, table_width: int) -> int:
    return _decode_workspace(batch, q_heads, *cache._sizes(), table_width)


def attn_decode_step(q, cache: KVCache, table, lens, *, scale: Optional[float] = None, out=None, lse=None,
                     workspace=None, stream=None):
    """ssm_attn_decode_step: one token per sequence, q [B, Hq, D], over its lens[b] cached tokens (the new one
    among them: write it first).  table [B, width] int32: the pages of each sequence; lens [B] int32.  scale defaults
    to 1 / sqrt(D).  workspace: attn_decode_workspace_bytes() bytes, allocated where not given.  Returns out
    [B, Hq, D]; an lse tensor [B, Hq] fp32 receives the log of the softmax sums."""
    if stream is None and workspace is None:
        r = (_native or _bound()).attn_decode_step(q, cache.address, cache.index, cache.is_bf16, table, lens, scale, out, lse)
        if r is not NotImplemented:
            return r
    call = _entry().attn_decode_step
    B, Hq, D = _three(q, "q")
    dev, dtype = cache.device, q.dtype
    cache.check_io(dtype)
    io = _io(q)
    if table.dim() != 2:
        raise ValueError(f"table must be [batch, width], got {tuple(table.shape)}")
    W = table.shape[1]
    shape = (B, Hq, cache.head_dim)
    vq = _view(q, "q", shape, dtype, dev)
    pt, pn = _index(table, "table", (B, W), _I32, dev), _index(lens, "lens", (B,), _I32, dev)
    if out is None:
        out, vo = _new(q, shape, stream)
    else:
        vo = _view(out, "out", shape, dtype, dev)
    pl = None if lse is None else _index(lse, "lse", (B, Hq), _F32, dev)
    pw, size = None, 0
    if workspace is None:
        size = _decode_workspace(B, Hq, *cache._sizes(), W)
        if size:
            workspace = _made(lambda: torch.empty(size, dtype=torch.uint8, device=dev), stream, dev, returned=False)
            pw = workspace.data_ptr()
    elif workspace.device != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {dev}")
    else:
        pw, size = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    buf = _Buffer()
    _two_views(buf, 0, *vq, *vo)
    at = ctypes.addressof(buf)
    st = call(B, Hq, io, D ** -0.5 if scale is None else scale, cache.address, at, pt, W, pn, at + _VIEW, pl, pw, size,
              stream_handle(stream, dev))
    if st != 0:
        _fail("ssm_attn_decode_step", st)
    return out
