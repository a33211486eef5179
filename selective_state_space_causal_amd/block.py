"""ctypes binding of the operators of include/ssm_block.h, which stand between a stack's residual stream and its mixers'
projections: the residual's addition and root-mean-square norm (in the io dtype or in 8 bits), weights in 4 bits, and
products of tokens with them.  Argument marshalling only: every step runs in the library's HIP kernels, there is no
fallback.

[T, D] tensors may be views with any row stride that is a multiple of 16 bytes; the D values of a row are contiguous."""
from __future__ import annotations

import ctypes
import warnings
from typing import NamedTuple, Optional

import torch

from . import _lib
from ._lib import SSM_BF16, SSM_F32, SsmError, _made, stream_handle

SSM_E4M3 = 2
GROUP = 32
MAX_WIDTH = 32768
MAX_FEATURES = 1 << 20
E4M3 = torch.float8_e4m3fn

_IO = {torch.float32: SSM_F32, torch.bfloat16: SSM_BF16}
_TOKENS = {**_IO, E4M3: SSM_E4M3}


class _Rows(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("stride", ctypes.c_int64)]


class _Q4(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("out_features", ctypes.c_int64),
                ("in_features", ctypes.c_int64)]


def declare(lib):
    """Argument types of the entry points (called once by _lib.load).  They came after the others, which they left as they
    were: a library of the same ABI version may be without them."""
    if not hasattr(lib, "ssm_q4_linear"):
        raise ImportError("libssm is of an earlier build, without the entry points of ssm_block.h; run python "
                          "selective_state_space_causal_amd/build.py")
    vp, i64, i32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t
    pr, pq = ctypes.POINTER(_Rows), ctypes.POINTER(_Q4)
    lib.ssm_rms_norm.restype = ctypes.c_int
    lib.ssm_rms_norm.argtypes = [i64, i64, i32, i32, i32, ctypes.c_float, pr, vp, pr, pr, pr, vp, vp]
    for name in ("ssm_q4_codes_bytes", "ssm_q4_scales_bytes"):
        getattr(lib, name).restype = sz
        getattr(lib, name).argtypes = [i64, i64]
    lib.ssm_q4_quantize.restype = ctypes.c_int
    lib.ssm_q4_quantize.argtypes = [i32, pr, pq, vp]
    lib.ssm_q4_dequantize.restype = ctypes.c_int
    lib.ssm_q4_dequantize.argtypes = [i32, pq, pr, vp]
    lib.ssm_q4_linear.restype = ctypes.c_int
    lib.ssm_q4_linear.argtypes = [i64, i32, i32, pr, vp, pq, pr, vp]


def _fail(name, st):
    raise SsmError(name, st, _lib.load().ssm_status_str(st).decode())


_native = None  # the usual case of the calls below, natively (csrc/block_binding.cpp); NotImplemented for any other


class _NoNative:
    """Every case goes through this file."""

    @staticmethod
    def _not_usual(*args):
        return NotImplemented
    rms_norm = q4_linear = q4_quantize = q4_dequantize = _not_usual


def _bound():
    global _native
    if _native is None:
        lib = _lib.load()
        try:
            from . import _block_fast
            _block_fast.bind(lib.ssm_abi_version(), *(ctypes.cast(getattr(lib, n), ctypes.c_void_p).value for n in (
                "ssm_rms_norm", "ssm_q4_linear", "ssm_q4_quantize", "ssm_q4_dequantize")), _fail)
            _native = _block_fast
        except ImportError as e:
            warnings.warn(f"the block calls' native binding is not built for this library ({e}): small calls are slower; run "
                          "selective_state_space_causal_amd/build.py")
            _native = _NoNative
    return _native


def _io(t: torch.Tensor, name: str) -> int:
    code = _IO.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} must be float32 or bfloat16, got {t.dtype}")
    return code


def _two(t: torch.Tensor, name: str):
    if t.dim() != 2:
        raise ValueError(f"{name} must be [tokens, width], got {tuple(t.shape)}")
    return t.shape


def _rows(t: torch.Tensor, name: str, shape, dtype, device):
    """A [T, D] tensor as rows, checked for shape, dtype, GPU device and contiguous rows."""
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if t.device != device or not t.is_cuda:
        raise ValueError(f"{name} must be on {device} (a GPU)")
    stride, one = t.stride()
    if one != 1 and shape[1] != 1:
        raise ValueError(f"{name}: the values of a row must be contiguous (stride {one})")
    # the stride of an axis of length 1 is never used, and torch leaves it arbitrary
    return _Rows(t.data_ptr(), stride if shape[0] > 1 else 0)


def _vector(t: torch.Tensor, name: str, n: int, device):
    if tuple(t.shape) == (n,) and t.dtype == torch.float32 and t.device == device and t.is_cuda and t.is_contiguous():
        return t.data_ptr()
    raise ValueError(f"{name} must be a contiguous float32 tensor of shape {(n,)} on {device} (a GPU), got {t.dtype} "
                     f"{tuple(t.shape)} on {t.device}")


def _call(entry, *args, stream, device):
    """The entry point's status.  It launches on the current device: the tensors' own, whichever that was before."""
    with torch.cuda.device(device):
        return entry(*args, stream_handle(stream, device))


def _empty(shape, dtype, device, stream):
    return _made(lambda: torch.empty(shape, dtype=dtype, device=device), stream, device)


# ---------------------------------------------------------------- the residual norm

def rms_norm(x, weight, *, residual=None, residual_out=None, eps: float = 1e-5, out_dtype=None, out=None, scale=None,
             stream=None):
    """ssm_rms_norm: y = h / sqrt(mean(h^2) + eps) * weight for each row of x [T, D], weight [D] fp32, with h = x, or
    x + residual [T, D] (x's dtype or fp32), which is rounded to residual's dtype and stored in residual_out (in place, in
    residual itself, where not given).  Returns y in x's dtype; with out_dtype=torch.float8_e4m3fn (codes, scale):
    codes [T, D] and scale [T] fp32, y = codes * scale.  out (pass x for in place, x's dtype only) and scale are made
    where not given."""
    if stream is None:
        r = (_native or _bound()).rms_norm(x, weight, residual, residual_out, eps, out_dtype, out, scale)
        if r is not NotImplemented:
            return r
    lib = _lib.load()
    T, D = shape = _two(x, "x")
    dev, dtype = x.device, x.dtype
    io = _io(x, "x")
    if out_dtype is None:
        out_dtype = dtype if out is None else out.dtype
    if out_dtype not in (dtype, E4M3):
        raise TypeError(f"the norm's output is of x's dtype or float8_e4m3fn, got {out_dtype}")
    q8 = out_dtype == E4M3
    if not q8 and scale is not None:
        raise ValueError("scale is for an output in float8_e4m3fn")
    if residual is None and residual_out is not None:
        raise ValueError("residual_out without residual")
    vx, pw = _rows(x, "x", shape, dtype, dev), _vector(weight, "weight", D, dev)
    vr = vro = None
    rio = io
    if residual is not None:
        rio = _io(residual, "residual")
        if residual.dtype not in (dtype, torch.float32):
            raise TypeError(f"residual must be {dtype} or float32, got {residual.dtype}")
        vr = _rows(residual, "residual", shape, residual.dtype, dev)
        vro = vr if residual_out is None else _rows(residual_out, "residual_out", shape, residual.dtype, dev)
    if out is None:
        out = _empty(shape, out_dtype, dev, stream)
    vo = _rows(out, "out", shape, out_dtype, dev)
    ps = None
    if q8:
        if scale is None:
            scale = _empty((T,), torch.float32, dev, stream)
        ps = _vector(scale, "scale", T, dev)
    st = _call(lib.ssm_rms_norm, T, D, io, rio, _TOKENS[out_dtype], eps, vx, pw, vr, vro, vo, ps, stream=stream, device=dev)
    if st != 0:
        _fail("ssm_rms_norm", st)
    return (out, scale) if q8 else out


# ---------------------------------------------------------------- weights in 4 bits

class Q4Weight(NamedTuple):
    """A weight [out_features, in_features] in 4 bits with a power of two for each 32 values of a row: codes uint8
    [ceil(out / 16), ceil(in / 128), 64, 16] and scales uint8 [ceil(out / 16), ceil(in / 512), 64, 4], laid out as
    include/ssm_block.h says.  q4_quantize makes one; pack() one from codes and scales in rows."""
    codes: torch.Tensor
    scales: torch.Tensor
    out_features: int
    in_features: int

    @classmethod
    def allocate(cls, out_features: int, in_features: int, device="cuda"):
        """One with uninitialised contents."""
        _check_features(out_features, in_features)
        codes, scales = _q4_shapes(out_features, in_features)
        return cls(torch.empty(codes, dtype=torch.uint8, device=device), torch.empty(scales, dtype=torch.uint8, device=device),
                   out_features, in_features)

    @classmethod
    def pack(cls, codes, scales):
        """From codes [M, K] uint8 (0 .. 15: sign, two bits of exponent, one of mantissa) and scales [M, ceil(K / 32)]
        uint8 (127 + the exponent of two, 2 .. 252; 255: the group is NaN), in rows, on any device."""
        if codes.dim() != 2 or codes.dtype != torch.uint8 or scales.dtype != torch.uint8:
            raise ValueError("codes must be [out_features, in_features] uint8, and scales uint8")
        (M, K), dev = codes.shape, codes.device
        _check_features(M, K)
        if tuple(scales.shape) != (M, -(-K // GROUP)) or scales.device != dev:
            raise ValueError(f"scales: {tuple(scales.shape)} on {scales.device}, expected {(M, -(-K // GROUP))} on {dev}")
        (mt, kt, _, _), (_, k4, _, _) = _q4_shapes(M, K)
        c = torch.zeros(mt * 16, kt * 128, dtype=torch.uint8, device=dev)
        c[:M, :K] = codes & 15
        c = c[:, 0::2] | c[:, 1::2] << 4
        s = torch.full((mt * 16, k4 * 16), 127, dtype=torch.uint8, device=dev)
        s[:M, :scales.shape[1]] = scales
        return cls(c.view(mt, 16, kt, 4, 16).permute(0, 2, 3, 1, 4).reshape(mt, kt, 64, 16).contiguous(),
                   s.view(mt, 16, k4, 4, 4).permute(0, 2, 4, 1, 3).reshape(mt, k4, 64, 4).contiguous(), M, K)

    def rows(self, start: int, stop: int) -> "Q4Weight":
        """Rows start .. stop - 1, sharing the memory; both multiples of 16 (or stop the end)."""
        if not 0 <= start < stop <= self.out_features or start % 16 or (stop % 16 and stop != self.out_features):
            raise ValueError(f"rows {start} .. {stop} of {self.out_features}: a part starts and ends at multiples of 16")
        tiles = slice(start // 16, -(-stop // 16))
        return Q4Weight(self.codes[tiles], self.scales[tiles], stop - start, self.in_features)

    @property
    def shape(self):
        """The weight's own shape, as a tensor's."""
        return torch.Size((self.out_features, self.in_features))


def _check_features(M, K):
    if not (1 <= M <= MAX_FEATURES and 16 <= K <= MAX_FEATURES and K % 16 == 0 and M * K <= 1 << 38):
        raise ValueError(f"a 4-bit weight has 1 to {MAX_FEATURES} rows of a multiple of 16 up to {MAX_FEATURES} values, at most 2^38 in all; "
                         f"got [{M}, {K}]")


def _q4_shapes(M, K):
    return (-(-M // 16), -(-K // 128), 64, 16), (-(-M // 16), -(-K // 512), 64, 4)


def _q4(w: Q4Weight, device):
    _check_features(w.out_features, w.in_features)
    for t, name, shape in zip(w, ("codes", "scales"), _q4_shapes(w.out_features, w.in_features)):
        if tuple(t.shape) != shape or t.dtype != torch.uint8 or t.device != device or not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous uint8 tensor of shape {shape} on {device} (a GPU), got {t.dtype} "
                             f"{tuple(t.shape)} on {t.device}")
    return _Q4(w.codes.data_ptr(), w.scales.data_ptr(), w.out_features, w.in_features)


def q4_quantize(w, *, out: Optional[Q4Weight] = None, stream=None) -> Q4Weight:
    """ssm_q4_quantize: w [out_features, in_features] (float32 or bfloat16) in 4 bits."""
    if stream is None and out is None:
        r = (_native or _bound()).q4_quantize(w)
        if r is not NotImplemented:
            return Q4Weight(*r, *w.shape)
    lib = _lib.load()
    M, K = _two(w, "w")
    io, dev = _io(w, "w"), w.device
    _check_features(M, K)
    vw = _rows(w, "w", w.shape, w.dtype, dev)
    if out is None:
        shapes = _q4_shapes(M, K)
        out = Q4Weight(*(_empty(s, torch.uint8, dev, stream) for s in shapes), M, K)
    elif (out.out_features, out.in_features) != (M, K):
        raise ValueError(f"out is a weight of {tuple(out.shape)}, expected {(M, K)}")
    st = _call(lib.ssm_q4_quantize, io, vw, _q4(out, dev), stream=stream, device=dev)
    if st != 0:
        _fail("ssm_q4_quantize", st)
    return out


def q4_dequantize(w: Q4Weight, *, dtype=None, out=None, stream=None):
    """ssm_q4_dequantize: the weight [out_features, in_features] in dtype (out's where given, else bfloat16; exact in both)."""
    if stream is None:
        r = (_native or _bound()).q4_dequantize(w, dtype, out)
        if r is not NotImplemented:
            return r
    lib = _lib.load()
    if dtype is None:
        dtype = torch.bfloat16 if out is None else out.dtype
    if dtype not in _IO:
        raise TypeError(f"a weight is read back as float32 or bfloat16, got {dtype}")
    dev = w.codes.device
    q = _q4(w, dev)
    if out is None:
        out = _empty(w.shape, dtype, dev, stream)
    st = _call(lib.ssm_q4_dequantize, _IO[dtype], q, _rows(out, "out", w.shape, dtype, dev), stream=stream, device=dev)
    if st != 0:
        _fail("ssm_q4_dequantize", st)
    return out


def q4_linear(x, w: Q4Weight, *, x_scale=None, out_dtype=None, out=None, stream=None):
    """ssm_q4_linear: x [T, in_features] times the weight's transpose, [T, out_features].  x is float32, bfloat16, or
    float8_e4m3fn with x_scale [T] fp32 (rms_norm gives both).  out_dtype: that of out where given, else x's, bfloat16
    for 8-bit tokens."""
    if stream is None:
        r = (_native or _bound()).q4_linear(x, w, x_scale, out_dtype, out)
        if r is not NotImplemented:
            return r
    lib = _lib.load()
    T, _ = _two(x, "x")
    dev = x.device
    if x.dtype not in _TOKENS:
        raise TypeError(f"x must be float32, bfloat16 or float8_e4m3fn, got {x.dtype}")
    if out_dtype is None:
        out_dtype = out.dtype if out is not None else torch.bfloat16 if x.dtype == E4M3 else x.dtype
    if out_dtype not in _IO:
        raise TypeError(f"the output is float32 or bfloat16, got {out_dtype}")
    if (x_scale is None) != (x.dtype != E4M3):
        raise ValueError("x_scale goes with float8_e4m3fn tokens")
    q = _q4(w, dev)
    vx = _rows(x, "x", (T, w.in_features), x.dtype, dev)
    ps = None if x_scale is None else _vector(x_scale, "x_scale", T, dev)
    shape = (T, w.out_features)
    if out is None:
        out = _empty(shape, out_dtype, dev, stream)
    vo = _rows(out, "out", shape, out_dtype, dev)
    st = _call(lib.ssm_q4_linear, T, _TOKENS[x.dtype], _IO[out_dtype], vx, ps, q, vo, stream=stream, device=dev)
    if st != 0:
        _fail("ssm_q4_linear", st)
    return out


# ---------------------------------------------------------------- a block's way in and out

def block_input(hidden, norm=None, residual=None, *, eps: float = 1e-5, tokens_8bit: bool = False, out=None, scale=None,
                stream=None):
    """What a block's first projection reads, as (tokens, scale or None): hidden [T, d_model] itself, or with norm (fp32
    [d_model]) its norm, after hidden has been added to the residual stream where one is given; tokens_8bit: in
    float8_e4m3fn with their scales, for a weight in 4 bits."""
    if norm is None:
        if residual is not None or tokens_8bit:
            raise ValueError("residual and tokens_8bit go with norm")
        return hidden, None
    y = rms_norm(hidden, norm, residual=residual, eps=eps, out_dtype=E4M3 if tokens_8bit else None, out=out, scale=scale,
                 stream=stream)
    return y if tokens_8bit else (y, None)


def check_weight(w, name, shape, dtype, device):
    """Refuses a projection's weight (a tensor or a Q4Weight) that is not [out, in] `shape`, of `dtype` and on `device`."""
    if tuple(w.shape) != tuple(shape):
        raise ValueError(f"{name} weight is {tuple(w.shape)}, expected {tuple(shape)}")
    if isinstance(w, Q4Weight):
        _q4(w, device)
    elif w.dtype != dtype:
        raise TypeError(f"{name} weight is {w.dtype}, expected {dtype}")
    elif w.device != device:
        raise ValueError(f"{name} weight is on {w.device}, expected {device}")


def project(x, w, x_scale=None):
    """x [T, K] times the transpose of w [M, K]: a Q4Weight (q4_linear), or a tensor of x's dtype (a plain library GEMM)."""
    if isinstance(w, Q4Weight):
        return q4_linear(x, w, x_scale=x_scale)
    if x_scale is not None:
        raise ValueError("8-bit tokens need a weight in 4 bits")
    return torch.nn.functional.linear(x, w)
