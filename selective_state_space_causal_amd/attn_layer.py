"""One rank's attention block of a hybrid stack (attention blocks between selective-SSM mixers), over packed
prompts and for one decoded token per sequence, composed from the operators of attn.py:

  qkv     = hidden @ qkv weight^T     [T, d_model] -> [T, Hq + 2 Hkv, D], q, k, v heads side by side
  q, k    rotated in place, k and v into the paged cache, in one launch (kv_write)
  o       = attn_prefill of the fresh keys, or of the cache's rows read back (kv_read) for a prompt's next
            chunk; attn_decode_step for a decoded token
  out     = o @ out weight^T          [T, Hq D] -> [T, d_model], the rank's partial sum

As with the mixer (layer.py), more than one rank adds its partial outputs outside this library.  The two
projections are plain library GEMMs (torch.nn.functional.linear), or q4_linear (block.py) where a weight is a
Q4Weight: both sides are token-major, a layout that the mixer's projections do not have over a prompt.  (For one token per
sequence the layouts coincide, and a caller that keeps a Projector can run its two projections around attn.py's calls
instead.)

With a norm the block takes the stack's residual stream: hidden (the last block's output) is added to it, and the
block runs on its norm, in 8 bits for weights in 4 bits where asked (rms_norm).  A call that is refused for what is missing, or of
another size, type or device, has left the stream as it was.

A mixer layer's hidden is [B, L, d_model]; hidden.view(-1, d_model) with row ends at multiples of L is the packed
form of the same tokens.
"""
from __future__ import annotations

import math

import torch

from . import attn
from .block import Q4Weight, block_input, check_weight, project


def cache_slots(table, seq, positions, page_size: int):
    """Slots of tokens: token i is at `positions[i]` of sequence `seq[i]`, whose pages are table[seq[i]] (int32
    [batch, width]).  -1 where there is no page (kv_write skips it).  int64, on table's device."""
    width = table.shape[1]
    if width == 0:  # nothing to look up
        return torch.full_like(positions, -1)
    at = positions.div(page_size, rounding_mode="floor")
    page = table[seq, at.clamp(0, width - 1)].long()
    held = (at >= 0) & (at < width) & (page >= 0)
    return torch.where(held, page * page_size + positions % page_size, -1)


def _check(hidden, weights, q_heads, cache, freq, mscale, *index):
    """Refuses what the calls after the norm would, by its presence, sizes, types and devices: it comes before hidden goes into the
    residual stream, so that a call that is put right and made again does not add it twice.  index: (name, tensor, shape,
    dtype) of each tensor of slots, positions, lengths and pages."""
    Hkv, D, P, dev = cache.kv_heads, cache.head_dim, cache.page_size, hidden.device
    check_weight(weights["qkv"], "qkv", ((q_heads + 2 * Hkv) * D, hidden.shape[1]), hidden.dtype, dev)
    check_weight(weights["out"], "out", (weights["out"].shape[0], q_heads * D), hidden.dtype, dev)
    cache.check_io(hidden.dtype)
    if cache.device != dev:
        raise ValueError(f"the cache is on {cache.device}, expected {dev}")
    if not 1 <= q_heads <= attn.MAX_HEADS or Hkv < 1 or q_heads % Hkv or not 8 <= D <= attn.MAX_HEAD_DIM or D % 8:
        raise ValueError(f"{q_heads} heads of {D} over {Hkv}: up to {attn.MAX_HEADS} heads, a multiple of the cache's, of a multiple of 8 up "
                         f"to {attn.MAX_HEAD_DIM}")
    if cache.pages < 1 or not attn.MIN_PAGE <= P <= attn.MAX_PAGE or P & (P - 1):
        raise ValueError(f"a cache has pages of a power of two from {attn.MIN_PAGE} to {attn.MAX_PAGE}, got {cache.pages} of {P}")
    pairs = freq.numel()
    if not (1 <= pairs <= D // 2 and math.isfinite(mscale)):
        raise ValueError(f"freq has {pairs} pairs and mscale is {mscale}: 1 to {D // 2} pairs, a finite mscale")
    for name, t, shape, dtype in (("freq", freq, (pairs,), torch.float64), *index):
        attn._index(t, name, shape, dtype, dev)


def _heads(hidden, weights, q_heads, cache, norm, residual, eps, tokens_8bit, check):
    """(q, k, v): views into one packed projection.  check(): what is refused before hidden goes into the residual stream."""
    Hkv, D = cache.kv_heads, cache.head_dim
    if tuple(weights["qkv"].shape) != ((q_heads + 2 * Hkv) * D, hidden.shape[1]):
        raise ValueError(f"qkv weight is {tuple(weights['qkv'].shape)}, expected {((q_heads + 2 * Hkv) * D, hidden.shape[1])}")
    if tokens_8bit and not isinstance(weights["qkv"], Q4Weight):
        raise ValueError("8-bit tokens need a weight in 4 bits")
    if residual is not None:
        check()
    x, scale = block_input(hidden, norm, residual, eps=eps, tokens_8bit=tokens_8bit)
    x = project(x, weights["qkv"], scale).view(x.shape[0], q_heads + 2 * Hkv, D)
    return x[:, :q_heads], x[:, q_heads:q_heads + Hkv], x[:, q_heads + Hkv:]


def attn_block_prefill(hidden, weights: dict, q_heads: int, cache: "attn.KVCache", slots, cu_q, positions, freq, *,
                       interleaved: bool = False, mscale: float = 1.0, context_slots=None, cu_k=None, norm=None,
                       residual=None, eps: float = 1e-5, tokens_8bit: bool = False):
    """hidden [T, d_model]: the new tokens of all sequences, packed (cu_q, int32 [batch + 1]), at cache rows `slots`
    and `positions` [T] int64; freq and mscale as rope_frequencies gives them.  weights: "qkv" [(Hq + 2 Hkv) D,
    d_model] and "out" [d_model, Hq D], each a tensor or a Q4Weight.  norm (fp32 [d_model]), residual [T, d_model] (updated
    in place), eps and tokens_8bit: as block_input takes them.  Sequences that already have cached tokens: context_slots are the
    slots of all of each sequence's tokens, the new ones last, packed by cu_k (both or neither).  Returns [T, d_model]."""
    if (context_slots is None) != (cu_k is None):
        raise ValueError("context_slots and cu_k go together")

    def check():
        T = hidden.shape[0]
        if cu_q.dim() != 1 or not 2 <= cu_q.shape[0] <= attn.MAX_BATCH + 1:
            raise ValueError(f"cu_q must be [batch + 1] with a batch of 1 to {attn.MAX_BATCH}, got {tuple(cu_q.shape)}")
        context = () if cu_k is None else (("context_slots", context_slots, (context_slots.numel(),), torch.int64),
                                           ("cu_k", cu_k, cu_q.shape, torch.int32))
        _check(hidden, weights, q_heads, cache, freq, mscale, ("slots", slots, (T,), torch.int64),
               ("positions", positions, (T,), torch.int64), ("cu_q", cu_q, cu_q.shape, torch.int32), *context)
    q, k, v = _heads(hidden, weights, q_heads, cache, norm, residual, eps, tokens_8bit, check)
    attn.kv_write(k, v, cache, slots, q=q, positions=positions, freq=freq, interleaved=interleaved, mscale=mscale, q_out=q,
                  k_out=k)
    if context_slots is not None:
        k, v = attn.kv_read(cache, context_slots, dtype=hidden.dtype)
    o = attn.attn_prefill(q, k, v, cu_q, cu_k)
    return project(o.flatten(1), weights["out"])


def attn_block_decode(hidden_t, weights: dict, q_heads: int, cache: "attn.KVCache", table, lens, freq, *,
                      interleaved: bool = False, mscale: float = 1.0, workspace=None, norm=None, residual=None,
                      eps: float = 1e-5, tokens_8bit: bool = False):
    """One token per sequence: hidden_t [B, d_model]; lens [B] int32 counts the sequence's tokens with the new one,
    which goes to position lens - 1 (a sequence of length 0 has none: nothing is written, its attention is
    zero).  table [B, width] int32.  norm, residual [B, d_model], eps and tokens_8bit as for a prompt.  Returns [B, d_model]."""
    def check():
        B = hidden_t.shape[0]
        if table.dim() != 2 or table.shape[1] < 1 or not 1 <= B <= attn.MAX_BATCH:
            raise ValueError(f"table must be [batch, width] with a batch of 1 to {attn.MAX_BATCH}, got {tuple(table.shape)} for {B} tokens")
        _check(hidden_t, weights, q_heads, cache, freq, mscale, ("table", table, (B, table.shape[1]), torch.int32),
               ("lens", lens, (B,), torch.int32))
        if workspace is not None:
            need, size = attn.attn_decode_workspace_bytes(B, q_heads, cache, table.shape[1]), workspace.numel() * workspace.element_size()
            if workspace.device != cache.device or not workspace.is_contiguous() or size < need or (need and workspace.data_ptr() % 16):
                raise ValueError(f"workspace must be a contiguous tensor of {need} bytes on {cache.device}, aligned to 16; got {size} on "
                                 f"{workspace.device}")
    q, k, v = _heads(hidden_t, weights, q_heads, cache, norm, residual, eps, tokens_8bit, check)
    positions = lens.long() - 1
    slots = cache_slots(table, torch.arange(table.shape[0], device=table.device), positions, cache.page_size)
    attn.kv_write(k, v, cache, slots, q=q, positions=positions, freq=freq, interleaved=interleaved, mscale=mscale, q_out=q)
    o = attn.attn_decode_step(q, cache, table, lens, workspace=workspace)
    return project(o.flatten(1), weights["out"])
