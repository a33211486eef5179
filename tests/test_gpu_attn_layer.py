"""An attention block after a mixer layer, on the GPU against fp64: packed prompts, a prompt in two chunks through the
quantised cache, and decoded tokens, each step resuming from the cache that the last one left."""
import numpy as np
import pytest
import torch

import selective_state_space_causal_amd as ssm
from oracle import attn as O
from selective_state_space_causal_amd import attn_layer as AL
from selective_state_space_causal_amd import inputs as I
from selective_state_space_causal_amd import layer
from tests.gpu_common import DEV, assert_close, f64, note

pytestmark = pytest.mark.gpu
TAU = 2e-2  # bf16 io, as for the mixer layer
HQ, HKV, D, PAGE = 8, 2, 64, 16


def bf16(x):
    return torch.from_numpy(np.asarray(x)).to(torch.bfloat16).to(torch.float64).numpy()


def block_weights(d_model, seed):
    g = torch.Generator().manual_seed(seed)
    n = (HQ + 2 * HKV) * D
    return {"qkv": (torch.randn(n, d_model, generator=g) * d_model ** -0.5).to(torch.bfloat16),
            "out": (torch.randn(d_model, HQ * D, generator=g) * (HQ * D) ** -0.5).to(torch.bfloat16)}


class Reference:
    """The block in fp64, rounded to bf16 where the block stores bf16; keys and values per sequence, as cached."""

    def __init__(self, w, freq, mscale, kind):
        self.qkv, self.out, self.freq, self.mscale, self.kind = f64(w["qkv"]), f64(w["out"]), freq, mscale, kind
        self.k, self.v = {}, {}

    def heads(self, hidden, pos):
        x = bf16(f64(hidden) @ self.qkv.T).reshape(len(pos), -1, D)
        q, k, v = x[:, :HQ], x[:, HQ:HQ + HKV], x[:, HQ + HKV:]
        return (bf16(O.rope(t, pos, self.freq, False, self.mscale)) for t in (q, k)), v

    def cached(self, x):
        if self.kind == "io":
            return x
        code, scale = O.quantize(x, self.kind)
        return code * scale[..., None].astype(np.float64)

    def append(self, b, k, v):
        for d, x in ((self.k, k), (self.v, v)):
            d[b] = np.concatenate([d.get(b, np.zeros((0, HKV, D))), self.cached(x)])

    def rows(self, b, q, k, v):
        """Attention of q [n, HQ, D], the last n tokens of k, v; through the out projection."""
        n = len(q)
        o = O.prefill(q, k, v, [0, n], [0, len(k)], True, D ** -0.5)[0]
        return bf16(bf16(o).reshape(n, -1) @ self.out.T)


@pytest.mark.parametrize("kind", ["e4m3", "int8", "io"])
def test_hybrid_stack(kind):
    note(f"hybrid stack, cache {kind}")
    w = I.LAYERS["layer_small"]
    L, B = 40, 2
    prm = I.make_params_distinct(w.d_inner, w.d_state)
    wts = I.make_proj_weights(w.d_model, w.d_inner, w.dt_rank, w.d_state, w.io)
    hidden = I.make_hidden(B, L, w.d_model, w.io)
    wd = {k: v.to(DEV) for k, v in wts.items()}
    pd = {k: (None if v is None else v.to(DEV)) for k, v in prm.items()}
    pj = ssm.Projector(DEV)
    x, _, _ = layer.mixer_prefill(hidden.to(DEV), wd, pd, pj)  # [B, L, d_model], tested elsewhere: the block's input
    pj.close()
    x = (x + hidden.to(DEV)).view(B * L, -1)

    bw = block_weights(w.d_model, 50)
    bd = {k: v.to(DEV) for k, v in bw.items()}
    freq, ms = ssm.rope_frequencies(D, scaling="yarn", factor=2.0, device=DEV)
    dtype = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8, "io": torch.bfloat16}[kind]
    cache = ssm.KVCache.allocate(12, PAGE, HKV, D, dtype, DEV)
    table = torch.tensor([[7, 2, 9, 4], [1, 11, 0, 5]], dtype=torch.int32, device=DEV)
    ref = Reference(bw, f64(freq), ms, kind)

    # first chunk: 30 tokens of the first row, 22 of the second; then the rest, over the cache
    cut = [30, 22]
    for part in range(2):
        lens = cut if part == 0 else [L - c for c in cut]
        start = [0, 0] if part == 0 else cut
        seq = torch.cat([torch.full((n,), b) for b, n in enumerate(lens)]).to(DEV)
        pos = torch.cat([torch.arange(s, s + n) for s, n in zip(start, lens)]).to(DEV)
        h = x[seq * L + pos].contiguous()
        cu = torch.tensor([0, lens[0], sum(lens)], dtype=torch.int32, device=DEV)
        slots = AL.cache_slots(table, seq, pos, PAGE)
        more = {}
        if part:
            allseq = torch.arange(B, device=DEV).repeat_interleave(L)
            allpos = torch.arange(L, device=DEV).repeat(B)
            more = dict(context_slots=AL.cache_slots(table, allseq, allpos, PAGE),
                        cu_k=torch.tensor([0, L, 2 * L], dtype=torch.int32, device=DEV))
        out = AL.attn_block_prefill(h, bd, HQ, cache, slots, cu, pos, freq, mscale=ms, **more)
        (q, k), v = ref.heads(h, f64(pos))
        want, at = [], 0
        for b, n in enumerate(lens):
            rows = slice(at, at + n)
            ref.append(b, k[rows], v[rows])
            # the cache's values in the io dtype for a second chunk, the fresh ones for the first
            kk, vv = (bf16(ref.k[b]), bf16(ref.v[b])) if part else (k[rows], v[rows])
            want.append(ref.rows(b, q[rows], kk, vv))
            at += n
        assert_close(out, np.concatenate(want), TAU, f"chunk {part} out", exact_inputs=False)

    # decoded tokens, one of the sequences ending after the second step
    for step in range(4):
        n = torch.tensor([L + step + 1, L + step + 1 if step < 2 else 0], dtype=torch.int32, device=DEV)
        ht = I.make_hidden(B, 1, w.d_model, w.io, seed=60 + step)[:, 0].to(DEV)
        out = AL.attn_block_decode(ht, bd, HQ, cache, table, n, freq, mscale=ms)
        (q, k), v = ref.heads(ht, f64(n) - 1)
        want = np.zeros((B, w.d_model))
        for b in range(B):
            if int(n[b]) == 0:
                continue
            ref.append(b, k[b:b + 1], v[b:b + 1])
            want[b] = ref.rows(b, q[b:b + 1], ref.k[b], ref.v[b])[0]
        assert_close(out, want, TAU, f"decode out step {step}", exact_inputs=False)


def test_slots():
    table = torch.tensor([[3, 0, -1], [1, 2, 4]], dtype=torch.int32, device=DEV)
    seq, pos = torch.tensor([0, 0, 1, 0, 0, 1], device=DEV), torch.tensor([5, 16, 47, 33, -1, 48], device=DEV)
    assert AL.cache_slots(table, seq, pos, 16).tolist() == [53, 0, 79, -1, -1, -1]
