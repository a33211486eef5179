"""One rank's attention block of a hybrid stack (attention blocks between selective-SSM mixers), over packed
prompts and for one decoded token per sequence, composed from the operators of attn.py:

  qkv     = hidden @ qkv weight^T     [T, d_model] -> [T, Hq + 2 Hkv, D], q, k, v heads side by side
  q, k    rotated in place, k and v into the paged cache, in one launch (kv_write)
  o       = attn_prefill of the fresh keys, or of the cache's rows read back (kv_read) for a prompt's next
            chunk; attn_decode_step for a decoded token
  out     = o @ out weight^T          [T, Hq D] -> [T, d_model], the rank's partial sum

As with the mixer (layer.py), more than one rank adds its partial outputs outside this library.  The two
projections are plain library GEMMs (torch.nn.functional.linear): both sides are token-major, a layout that
the mixer's projections do not have over a prompt.  (For one token per sequence the layouts coincide, and a caller that
keeps a Projector can run its two projections around attn.py's calls instead.)

A mixer layer's hidden is [B, L, d_model]; hidden.view(-1, d_model) with row ends at multiples of L is the packed
form of the same tokens.
"""
from __future__ import annotations

import torch
from torch.nn.functional import linear

from . import attn


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


def _heads(x, weights, q_heads, cache):
    """(q, k, v): views into one packed projection."""
    Hkv, D = cache.kv_heads, cache.head_dim
    if weights["qkv"].shape[0] != (q_heads + 2 * Hkv) * D:
        raise ValueError(f"qkv weight has {weights['qkv'].shape[0]} rows, expected {(q_heads + 2 * Hkv) * D}")
    x = linear(x, weights["qkv"]).view(x.shape[0], q_heads + 2 * Hkv, D)
    return x[:, :q_heads], x[:, q_heads:q_heads + Hkv], x[:, q_heads + Hkv:]


def attn_block_prefill(hidden, weights: dict, q_heads: int, cache: "attn.KVCache", slots, cu_q, positions, freq, *,
                       interleaved: bool = False, mscale: float = 1.0, context_slots=None, cu_k=None):
    """hidden [T, d_model]: the new tokens of all sequences, packed (cu_q, int32 [batch + 1]), at cache rows `slots`
    and `positions` [T] int64; freq and mscale as rope_frequencies gives them.  weights: "qkv" [(Hq + 2 Hkv) D,
    d_model] and "out" [d_model, Hq D].  Sequences that already have cached tokens: context_slots are the
    slots of all of each sequence's tokens, the new ones last, packed by cu_k (both or neither).  Returns [T, d_model]."""
    if (context_slots is None) != (cu_k is None):
        raise ValueError("context_slots and cu_k go together")
    q, k, v = _heads(hidden, weights, q_heads, cache)
    attn.kv_write(k, v, cache, slots, q=q, positions=positions, freq=freq, interleaved=interleaved, mscale=mscale, q_out=q,
                  k_out=k)
    if context_slots is not None:
        k, v = attn.kv_read(cache, context_slots, dtype=hidden.dtype)
    o = attn.attn_prefill(q, k, v, cu_q, cu_k)
    return linear(o.flatten(1), weights["out"])


def attn_block_decode(hidden_t, weights: dict, q_heads: int, cache: "attn.KVCache", table, lens, freq, *,
                      interleaved: bool = False, mscale: float = 1.0, workspace=None):
    """One token per sequence: hidden_t [B, d_model]; lens [B] int32 counts the sequence's tokens with the new one,
    which goes to position lens - 1 (a sequence of length 0 has none: nothing is written, its attention is
    zero).  table [B, width] int32.  Returns [B, d_model]."""
    q, k, v = _heads(hidden_t, weights, q_heads, cache)
    positions = lens.long() - 1
    slots = cache_slots(table, torch.arange(table.shape[0], device=table.device), positions, cache.page_size)
    attn.kv_write(k, v, cache, slots, q=q, positions=positions, freq=freq, interleaved=interleaved, mscale=mscale, q_out=q)
    o = attn.attn_decode_step(q, cache, table, lens, workspace=workspace)
    return linear(o.flatten(1), weights["out"])
