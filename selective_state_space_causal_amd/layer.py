"""One rank's slice of a selective-SSM mixer layer, over a prompt and for one decoded token,
composed from the library's
C-ABI calls (argument marshalling only; every step runs in the library's kernels or in its
hipBLASLt GEMMs):

  x, z    = in_proj (column shard)            [B, L, d_model] -> [B, D, L] each
  u       = conv + SiLU front                 [B, D, L]
  r, B, C = x_proj rows reading these channels [B, D, L] -> [B, L, R], [B, L, N], [B, L, N]
  dt      = dt_proj                           [B, L, R] -> [B, D, L]
  y, h, c = ssm_prefill                       (the scan; leaves the h / conv cache)
  out     = out_proj (row shard)              [B, D, L] -> [B, L, d_model], a partial sum

"Scaling State-Space Models on Multiple GPUs with Tensor Parallelism" (euno.news summary of
arXiv 2602.21144), Methodology items 1-2.  With more than one rank, x_proj's outputs and out
are partial sums that the ranks add (all-reduces that this library does not run); on one GPU the slice's
partials are used as they are.

Decode (mixer_decode_step) runs one token per batch row from the cache the prefill left:
in_proj, then either the four per-token stages as separate calls (conv_silu from the conv
cache, x_proj, dt_proj, ssm_decode_step) or the same four as ssm_decode_fused (two kernels),
then out_proj.

in_proj's shard is one [2D, d_model] weight whose first D rows make x and last D rows make z
(the mixer's packed input projection).  With one batch row, one GEMM writes [1, 2D, L] and x
and z are its two halves, each already a contiguous [1, D, L] tensor; otherwise the two halves
of the weight run as two GEMMs.  x_proj's rows are stacked likewise ([R + 2N, D]: low-rank, B,
C); for bf16 with D and L multiples of 8, the conv front and x_proj run as one fused kernel
(ssm_conv_xproj) and u is never stored; otherwise u is materialised and x_proj runs as three
GEMMs.  out is written in the io dtype by default (the partial that the 8-bit all-reduce codec
then quantizes); out_dtype=torch.float32 keeps it in fp32.

Weights in 4 bits: in_proj's and out_proj's weights ("in_xz", "in_x", "in_z", "out") may be Q4Weights (block.py).  A decoded
token is multiplied with them as they are (q4_linear); a prompt reads them back into the io dtype (q4_dequantize), since its
projections are in the mixer's own channel-major layouts.

With a norm the layer takes the stack's residual stream: hidden (the last block's output) is added to it, and in_proj
reads its norm, in 8 bits for a decoded token where asked (rms_norm).  A call that is refused for what is missing, or of another
size, type, device or alignment, has left the stream as it was.

Given a stream, a layer takes the memory of all that it makes from that stream's pool: a block of the current stream's may
still be in use by work queued there, which nothing orders before the layer's.
"""
from __future__ import annotations

import contextlib

import torch

from . import _lib
from .block import E4M3, Q4Weight, _check_features, _q4_shapes, block_input, q4_dequantize, q4_linear

CONV_W = 4


def _stacked_in_proj(hidden, weights) -> bool:
    """True when one GEMM can write x and z: a stacked weight, one batch row, and z's half
    starting on a 16-byte boundary."""
    if "in_xz" not in weights or hidden.shape[0] != 1:
        return False
    D, L = weights["in_xz"].shape[0] // 2, hidden.shape[1]
    return (D * L * hidden.element_size()) % 16 == 0


def _fused_conv_xproj(hidden, weights) -> bool:
    """True when the conv front and x_proj can run as one kernel: the stacked x_proj weight,
    bf16, and d_inner and seqlen multiples of 8."""
    D, L = weights["in_x"].shape[0], hidden.shape[1]
    return "x_all" in weights and hidden.dtype == torch.bfloat16 and D % 8 == 0 and L % 8 == 0


def _used(weights: dict, stacked: bool) -> tuple:
    """The projection weights that a call reads."""
    return ("in_xz", "out") if stacked else ("in_x", "in_z", "out")


def _on(stream):
    """With `stream` (None: as it is) current, for what is allocated."""
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


def _returned(tensors, stream, device):
    """Tensors of `stream`'s pool, for use on the current stream: not handed out again before that is done with them."""
    if stream is not None:
        for t in tensors:
            t.record_stream(torch.cuda.current_stream(device))
    return tensors


# What the stages after the norm would refuse is refused before hidden goes into the residual stream, so that a call that is put right
# and made again does not add it twice: what is missing, or of another size, type, device or alignment than they take.  (Tensors
# that share memory, and a seqlen of 2^24 or more, they refuse themselves, and memory may run out in one.  11 us of the host for a
# decode step.)

def _look(what, device):
    """what: (name, tensor, shape, dtype, bytes its address is a multiple of) of each."""
    index = device.index
    for name, t, shape, dtype, align in what:
        if t is not None and t.shape == shape and t.dtype == dtype and t.get_device() == index and t.is_contiguous() and not t.data_ptr() % align:
            continue
        _lib._check(t, name, shape, dtype, device)
        raise ValueError(f"{name} must be aligned to {align} bytes")


def _weights(weights: dict, shapes: dict, dtype):
    """The weights of those names as _look takes them."""
    for k, (shape, align) in shapes.items():
        w = weights[k]
        if not isinstance(w, Q4Weight):
            yield k, w, shape, dtype, align
            continue
        M, K = shape
        if (w.out_features, w.in_features) != shape:
            raise ValueError(f"{k} weight is {tuple(w.shape)}, expected {shape}")
        _check_features(M, K)
        codes, scales = _q4_shapes(M, K)
        yield k + " codes", w.codes, codes, torch.uint8, 16
        yield k + " scales", w.scales, scales, torch.uint8, 16


def _parameters(params: dict, D: int, N: int):
    f32 = torch.float32
    if not 1 <= N <= _lib.MAX_STATE:
        raise ValueError(f"d_state is {N}, up to {_lib.MAX_STATE}")
    p = [("A", params["A"], (D, N), f32, 16), ("Dskip", params["Dskip"], (D,), f32, 4), ("dt_bias", params["dt_bias"], (D,), f32, 4),
         ("conv_w", params["conv_w"], (D, CONV_W), f32, 16)]
    bias = params.get("conv_b")
    return p if bias is None else p + [("conv_b", bias, (D,), f32, 4)]


def _projector(proj):
    if proj is None or proj.handle is None:
        raise ValueError("a projector, not closed, is required")


def _check_prefill(hidden, weights: dict, params: dict, proj, b: dict):
    (B, L, DM), D, R, N = hidden.shape, weights["in_x"].shape[0], weights["x_dt"].shape[0], params["A"].shape[1]
    dt, f32, stacked, conv_xproj = hidden.dtype, torch.float32, "xz" in b, "u" not in b
    _projector(proj)
    shapes = dict(in_xz=((2 * D, DM), 16)) if stacked else dict(in_x=((D, DM), 16), in_z=((D, DM), 16))
    shapes.update(dict(x_all=((R + 2 * N, D), 16)) if conv_xproj else dict(x_dt=((R, D), 16), x_B=((N, D), 16), x_C=((N, D), 16)),
                  dt=((D, R), 16), out=((DM, D), 16))
    _lib._io_code(b["out"].dtype)
    rows = ("dt", "y") if conv_xproj else ("u", "dt", "y")
    _look((*_weights(weights, shapes, dt), *_parameters(params, D, N),
           *((("xz", b["xz"], (1, 2 * D, L), dt, 16),) if stacked else ()),
           *((k, b[k], (B, D, L), dt, 16) for k in ("x", "z", *rows)),
           *((k, b[k], (B, L, n), dt, 16) for k, n in (("lowrank", R), ("Bm", N), ("Cm", N))),
           ("h", b["h"], (B, D, N), f32, 16), ("c", b["c"], (B, D, CONV_W - 1), f32, 16), ("out", b["out"], (B, L, DM), b["out"].dtype, 16)),
          hidden.device)


def _check_decode(hidden_t, weights: dict, params: dict, proj, h, conv, b: dict, fused: bool):
    (B, DM), D, R, N = hidden_t.shape, weights["in_x"].shape[0], weights["x_dt"].shape[0], params["A"].shape[1]
    dt, dev, f32, stacked = hidden_t.dtype, hidden_t.device, torch.float32, "xz" in b
    es = dt.itemsize  # the fused step takes its weights and rows at any address
    shapes = dict(in_xz=((2 * D, DM), 16)) if stacked else dict(in_x=((D, DM), 16), in_z=((D, DM), 16))
    shapes["out"] = ((DM, D), 16)
    if not fused or not all(isinstance(weights[k], Q4Weight) for k in shapes):
        _projector(proj)
    if fused:
        shapes.update(x_all=((R + 2 * N, D), es), dt=((D, R), es))
    else:
        shapes.update(dict(x_all=((R + 2 * N, D), 16)) if "xo" in b else dict(x_dt=((R, D), 16), x_B=((N, D), 16), x_C=((N, D), 16)),
                      dt=((D, R), 16))
    _lib._io_code(b["out"].dtype)
    _look((*_weights(weights, shapes, dt), *_parameters(params, D, N), ("h", h, (B, D, N), f32, 16), ("conv", conv, (B, D, CONV_W - 1), f32, 4),
           *((("xz", b["xz"], (1, 2 * D, 1), dt, 16),) if stacked else ()),
           *((k, b[k], (B, D, 1), dt, es if stacked else 16) for k in ("x", "z")), ("y", b["y"], (B, D, 1), dt, 16),
           ("out", b["out"], (B, 1, DM), b["out"].dtype, 16)), dev)
    if fused:
        need, ws = _lib.decode_fused_workspace_bytes(B, D, R, N, dt), b["ws"]
        if need == 0:
            raise ValueError(f"the fused step takes no d_state of {N} with a rank of {R}")
        if ws.device != dev or not ws.is_contiguous() or ws.numel() * ws.element_size() < need:
            raise ValueError(f"ws must be a contiguous tensor of {need} bytes on {dev}")
        return
    _look((*((("xo", b["xo"], (1, 1, R + 2 * N), dt, 16),) if "xo" in b else ()), ("u", b["u"], (B, D, 1), dt, 16), ("dt", b["dt"], (B, D, 1), dt, 16),
           *((k, b[k], (B, 1, n), dt, es if "xo" in b and k != "lowrank" else 16) for k, n in (("lowrank", R), ("Bt", N), ("Ct", N)))), dev)


def alloc_buffers(hidden, weights: dict, d_state: int, out_dtype=None, normed: bool = False) -> dict:
    """Every tensor the layer writes, on hidden's device, from the current stream's memory."""
    B, L, DM = hidden.shape
    D = weights["in_x"].shape[0]
    R = weights["x_dt"].shape[0]
    dev, dt = hidden.device, hidden.dtype
    bufs = {}
    if _stacked_in_proj(hidden, weights):
        bufs["xz"] = torch.empty(B, 2 * D, L, dtype=dt, device=dev)
        bufs["x"], bufs["z"] = bufs["xz"][:, :D], bufs["xz"][:, D:]
    else:
        bufs["x"] = torch.empty(B, D, L, dtype=dt, device=dev)
        bufs["z"] = torch.empty_like(bufs["x"])
    for k in ("dt", "y") if _fused_conv_xproj(hidden, weights) else ("u", "dt", "y"):
        bufs[k] = torch.empty(B, D, L, dtype=dt, device=dev)
    bufs["lowrank"] = torch.empty(B, L, R, dtype=dt, device=dev)
    bufs["Bm"] = torch.empty(B, L, d_state, dtype=dt, device=dev)
    bufs["Cm"] = torch.empty(B, L, d_state, dtype=dt, device=dev)
    bufs["h"] = torch.empty(B, D, d_state, dtype=torch.float32, device=dev)
    bufs["c"] = torch.empty(B, D, CONV_W - 1, dtype=torch.float32, device=dev)
    bufs["out"] = torch.empty(B, L, DM, dtype=out_dtype or dt, device=dev)
    if normed:
        bufs["normed"] = torch.empty(B, L, DM, dtype=dt, device=dev)
    for k in _used(weights, "xz" in bufs):
        if isinstance(weights[k], Q4Weight):
            bufs["w_" + k] = torch.empty(weights[k].shape, dtype=dt, device=dev)
    return bufs


def stages(hidden, weights: dict, params: dict, proj: "_lib.Projector", bufs: dict, stream=None, norm=None, residual=None,
           eps: float = 1e-5):
    """The layer as a list of (stage name, call), in order; each call enqueues its kernels on
    `stream` and writes into `bufs`."""
    P, b = proj, bufs
    pre = []
    for k in _used(weights, "xz" in b):
        if isinstance(weights[k], Q4Weight):
            pre.append((k + "_weight", lambda w=weights[k], o=b["w_" + k]: q4_dequantize(w, out=o, stream=stream)))
            weights = {**weights, k: b["w_" + k]}
    if norm is not None:
        if residual is not None and residual.shape != hidden.shape:
            raise ValueError(f"residual: shape {tuple(residual.shape)}, expected {tuple(hidden.shape)}")
        x, hidden, DM = hidden, b["normed"], hidden.shape[2]

        def norm_stage():
            tokens, rows = x.view(-1, DM), None if residual is None else residual.view(-1, DM)
            if residual is not None:
                _check_prefill(x, weights, params, proj, b)
            block_input(tokens, norm, rows, eps=eps, out=b["normed"].view(-1, DM), stream=stream)
        pre.append(("norm", norm_stage))
    elif residual is not None:
        raise ValueError("residual goes with norm")
    if "xz" in b:
        st = pre + [("in_proj_xz", lambda: P(_lib.PROJ_IN, hidden, weights["in_xz"], out=b["xz"], stream=stream))]
    else:
        st = pre + [("in_proj_x", lambda: P(_lib.PROJ_IN, hidden, weights["in_x"], out=b["x"], stream=stream)),
                    ("in_proj_z", lambda: P(_lib.PROJ_IN, hidden, weights["in_z"], out=b["z"], stream=stream))]
    if "u" not in b:
        R = weights["x_dt"].shape[0]
        st.append(("conv_xproj", lambda: _lib.conv_xproj(b["x"], params, weights["x_all"], R, lowrank=b["lowrank"],
                                                         Bm=b["Bm"], Cm=b["Cm"], stream=stream)))
    else:
        st += [("conv_silu", lambda: _lib.conv_silu(b["x"], params, u=b["u"], stream=stream)),
               ("x_proj_dt", lambda: P(_lib.PROJ_X, b["u"], weights["x_dt"], out=b["lowrank"], stream=stream)),
               ("x_proj_B", lambda: P(_lib.PROJ_X, b["u"], weights["x_B"], out=b["Bm"], stream=stream)),
               ("x_proj_C", lambda: P(_lib.PROJ_X, b["u"], weights["x_C"], out=b["Cm"], stream=stream))]
    return st + [
        ("dt_proj", lambda: P(_lib.PROJ_DT, b["lowrank"], weights["dt"], out=b["dt"], stream=stream)),
        ("scan", lambda: _lib.prefill(b["x"], b["dt"], b["z"], b["Bm"], b["Cm"], params, y=b["y"], h_out=b["h"],
                                      conv_out=b["c"], stream=stream)),
        ("out_proj", lambda: P(_lib.PROJ_OUT, b["y"], weights["out"], out=b["out"], stream=stream)),
    ]


def mixer_prefill(hidden, weights: dict, params: dict, proj: "_lib.Projector", *, out_dtype=None, stream=None, norm=None,
                  residual=None, eps: float = 1e-5):
    """Returns (out [B, L, d_model] partial in out_dtype (default: hidden's dtype), h [B, D, N],
    conv [B, D, 3]).  norm (fp32 [d_model]): in_proj reads the norm of hidden, or with residual [B, L, d_model] (hidden's
    dtype or fp32, contiguous, updated in place) of its sum with hidden."""
    with _on(stream):
        bufs = alloc_buffers(hidden, weights, params["A"].shape[1], out_dtype, norm is not None)
        for _, call in stages(hidden, weights, params, proj, bufs, stream, norm, residual, eps):
            call()
    return _returned((bufs["out"], bufs["h"], bufs["c"]), stream, hidden.device)


# ---- decode: one token per batch row through the layer, from the cache ----

def alloc_decode_buffers(hidden_t, weights: dict, d_state: int, fused: bool, out_dtype=None, normed: bool = False,
                         tokens_8bit: bool = False) -> dict:
    """Every tensor a decode step writes besides the cache and the residual stream, on hidden_t's device, from the current
    stream's memory."""
    B, DM = hidden_t.shape
    D, R = weights["in_x"].shape[0], weights["x_dt"].shape[0]
    dev, dt = hidden_t.device, hidden_t.dtype
    b = {}
    if normed:
        b["normed"] = torch.empty(B, DM, dtype=E4M3 if tokens_8bit else dt, device=dev)
        if tokens_8bit:
            b["scale"] = torch.empty(B, dtype=torch.float32, device=dev)
    if B == 1 and "in_xz" in weights:
        b["xz"] = torch.empty(1, 2 * D, 1, dtype=dt, device=dev)
        b["x"], b["z"] = b["xz"][:, :D], b["xz"][:, D:]
    else:
        b["x"] = torch.empty(B, D, 1, dtype=dt, device=dev)
        b["z"] = torch.empty_like(b["x"])
    b["y"] = torch.empty(B, D, 1, dtype=dt, device=dev)
    b["out"] = torch.empty(B, 1, DM, dtype=out_dtype or dt, device=dev)
    if fused:
        b["ws"] = torch.empty(max(1, _lib.decode_fused_workspace_bytes(B, D, R, d_state, dt)), dtype=torch.uint8,
                              device=dev)
        return b
    b["u"] = torch.empty(B, D, 1, dtype=dt, device=dev)
    b["dt"] = torch.empty(B, D, 1, dtype=dt, device=dev)
    if B == 1 and "x_all" in weights:  # one GEMM writes [1, 1, R + 2N]: low-rank, B_t, C_t in a row
        b["xo"] = torch.empty(1, 1, R + 2 * d_state, dtype=dt, device=dev)
        b["lowrank"], b["Bt"], b["Ct"] = (b["xo"][:, :, :R], b["xo"][:, :, R:R + d_state],
                                          b["xo"][:, :, R + d_state:])
    else:
        b["lowrank"] = torch.empty(B, 1, R, dtype=dt, device=dev)
        b["Bt"] = torch.empty(B, 1, d_state, dtype=dt, device=dev)
        b["Ct"] = torch.empty(B, 1, d_state, dtype=dt, device=dev)
    return b


def decode_stages(hidden_t, weights: dict, params: dict, proj: "_lib.Projector", h, conv, bufs: dict,
                  fused: bool, stream=None, norm=None, residual=None, eps: float = 1e-5):
    """One decode step of the layer as a list of (stage name, call); h [B, D, N] and conv
    [B, D, 3] are updated in place.  Unfused: in_proj, conv_silu (from the conv cache), x_proj
    (one GEMM for one batch row with the stacked weight, else three), dt_proj, ssm_decode_step,
    out_proj.  Fused: in_proj, ssm_decode_fused, out_proj."""
    b = bufs
    B, DM = hidden_t.shape
    tokens, scale = (hidden_t, None) if norm is None else (b["normed"], b.get("scale"))
    hs = tokens.view(B, 1, DM)
    if scale is not None and not all(isinstance(weights[k], Q4Weight) for k in _used(weights, "xz" in b) if k != "out"):
        raise ValueError("8-bit tokens need in_proj's weight in 4 bits")

    def P(kind, x, w, *, out, stream):  # one token per row: the layouts of both sides are [B, features]
        if not isinstance(w, Q4Weight):
            return proj(kind, x, w, out=out, stream=stream)
        return q4_linear(x.view(B, -1), w, x_scale=scale if kind == _lib.PROJ_IN else None, out=out.view(B, -1), stream=stream)

    R = weights["x_dt"].shape[0]
    st = []
    if norm is not None:
        def norm_stage():
            if residual is not None:
                _check_decode(hidden_t, weights, params, proj, h, conv, b, fused)
            block_input(hidden_t, norm, residual, eps=eps, tokens_8bit=scale is not None, out=b["normed"], scale=scale, stream=stream)
        st.append(("norm", norm_stage))
    elif residual is not None:
        raise ValueError("residual goes with norm")
    if "xz" in b:
        st.append(("in_proj_xz", lambda: P(_lib.PROJ_IN, hs, weights["in_xz"], out=b["xz"], stream=stream)))
    else:
        st += [("in_proj_x", lambda: P(_lib.PROJ_IN, hs, weights["in_x"], out=b["x"], stream=stream)),
               ("in_proj_z", lambda: P(_lib.PROJ_IN, hs, weights["in_z"], out=b["z"], stream=stream))]
    x2, z2, y2 = b["x"].view(B, -1), b["z"].view(B, -1), b["y"].view(B, -1)
    if fused:
        st.append(("decode_fused", lambda: _lib.decode_fused(x2, z2, params, weights["x_all"], weights["dt"], R, h, conv,
                                                             y_t=y2, workspace=b["ws"], stream=stream)))
    else:
        st.append(("conv_silu", lambda: _lib.conv_silu(b["x"], params, conv, u=b["u"], stream=stream)))
        if "xo" in b:
            st.append(("x_proj", lambda: P(_lib.PROJ_X, b["u"], weights["x_all"], out=b["xo"], stream=stream)))
        else:
            st += [("x_proj_dt", lambda: P(_lib.PROJ_X, b["u"], weights["x_dt"], out=b["lowrank"], stream=stream)),
                   ("x_proj_B", lambda: P(_lib.PROJ_X, b["u"], weights["x_B"], out=b["Bt"], stream=stream)),
                   ("x_proj_C", lambda: P(_lib.PROJ_X, b["u"], weights["x_C"], out=b["Ct"], stream=stream))]
        st += [("dt_proj", lambda: P(_lib.PROJ_DT, b["lowrank"], weights["dt"], out=b["dt"], stream=stream)),
               ("decode_step", lambda: _lib.decode_step(x2, b["dt"].view(B, -1), z2, b["Bt"].view(B, -1),
                                                        b["Ct"].view(B, -1), params, h, conv, y_t=y2, stream=stream))]
    st.append(("out_proj", lambda: P(_lib.PROJ_OUT, b["y"], weights["out"], out=b["out"], stream=stream)))
    return st


def mixer_decode_step(hidden_t, weights: dict, params: dict, proj: "_lib.Projector", h, conv, *, fused: bool = True,
                      out_dtype=None, bufs=None, stream=None, norm=None, residual=None, eps: float = 1e-5,
                      tokens_8bit: bool = False):
    """One decoded token per batch row: hidden_t [B, d_model]; h [B, D, N] and conv [B, D, 3]
    (the cache) are updated in place.  Returns out [B, d_model], the layer's partial sum.
    fused needs the stacked x_proj weight ("x_all") and d_state 16.  norm and residual [B, d_model] as for mixer_prefill;
    tokens_8bit: the norm in 8 bits, for an in_proj in 4 bits (bufs are then made with normed and tokens_8bit)."""
    if tokens_8bit and norm is None:
        raise ValueError("tokens_8bit goes with norm")
    if bufs is not None and norm is not None and ("normed" not in bufs or ("scale" in bufs) != tokens_8bit):
        raise ValueError(f"bufs were not made with normed=True, tokens_8bit={tokens_8bit}")
    made = bufs is None
    with _on(stream):
        if made:
            bufs = alloc_decode_buffers(hidden_t, weights, params["A"].shape[1], fused, out_dtype, norm is not None, tokens_8bit)
        for _, call in decode_stages(hidden_t, weights, params, proj, h, conv, bufs, fused, stream, norm, residual, eps):
            call()
    if made:
        _returned((bufs["out"],), stream, hidden_t.device)
    return bufs["out"].view(hidden_t.shape[0], -1)
