"""Mixer layers and attention blocks on a residual stream, with projections in 4 bits, on the GPU: against the oracle's
composition (bf16 io: the tolerance of the layer's own tests), and call by call against the operators."""
import numpy as np
import pytest
import torch

import selective_state_space_causal_amd as ssm
from oracle import block as O
from oracle import proj as P
from selective_state_space_causal_amd import attn_layer as AL
from selective_state_space_causal_amd import block as B
from selective_state_space_causal_amd import inputs as I
from selective_state_space_causal_amd import layer
from tests.gpu_common import DEV, assert_close, f64, note

pytestmark = pytest.mark.gpu
TAU = 2e-2
E4M3 = torch.float8_e4m3fn
EPS = 1e-5


@pytest.fixture(scope="module")
def pj():
    p = ssm.Projector(DEV)
    yield p
    p.close()


def four_bit(wts):
    """(weights on the device with in_proj and out_proj in 4 bits, the same weights' values on the host)."""
    wd = {k: v.to(DEV) for k, v in wts.items()}
    D, R, N = wts["in_x"].shape[0], wts["x_dt"].shape[0], wts["x_B"].shape[0]
    wd["x_dt"], wd["x_B"], wd["x_C"] = wd["x_all"][:R], wd["x_all"][R:R + N], wd["x_all"][R + N:]
    for k in ("in_xz", "out"):
        wd[k] = ssm.q4_quantize(wd[k])
    wd["in_x"], wd["in_z"] = wd["in_xz"].rows(0, D), wd["in_xz"].rows(D, 2 * D)
    host = dict(wts)
    for k in ("in_x", "in_z", "out"):
        host[k] = ssm.q4_dequantize(wd[k]).cpu()
    return wd, host


def stream(x, res, dtype):
    """(the residual stream after x, as it is stored, and its norm's input in fp64)."""
    h = (x.float() + res.float()).to(dtype)
    return h, f64(h)


@pytest.mark.parametrize("rows", [1, 2])
@pytest.mark.parametrize("fused", [False, True])
@pytest.mark.parametrize("kind", ["plain", "norm", "e4m3"])
def test_mixer_on_a_residual_stream(pj, rows, fused, kind):
    """A prompt of 40 tokens, then 4 decoded ones, each layer's input the norm of the stream."""
    note(f"mixer in 4 bits, rows={rows} fused={fused} {kind}")
    w = I.LAYERS["layer_small"]
    L, steps, DM = 40, 4, w.d_model
    prm = I.make_params_distinct(w.d_inner, w.d_state)
    wd, host = four_bit(I.make_proj_weights(DM, w.d_inner, w.dt_rank, w.d_state, w.io))
    pd = {k: (None if v is None else v.to(DEV)) for k, v in prm.items()}
    hidden = I.make_hidden(rows, L + steps, DM, w.io)
    g = torch.Generator().manual_seed(1)
    norm = 1 + 0.2 * torch.randn(DM, generator=g)
    rdt = torch.bfloat16 if kind == "norm" else torch.float32
    res = (2 * torch.randn(rows, L + steps, DM, generator=g)).to(rdt)
    kw = {} if kind == "plain" else dict(norm=norm.to(DEV), eps=EPS)

    def reads(x, r):
        """What in_proj reads, and the stream; x [.., DM] on the host."""
        if kind == "plain":
            return x, None
        h, v = stream(x, r, rdt)
        y = O.rms_norm(v.reshape(-1, DM), norm.double().numpy(), EPS).reshape(v.shape)
        return torch.from_numpy(y).to(torch.bfloat16), h

    x, want_res = reads(hidden[:, :L], res[:, :L])
    r = res[:, :L].contiguous().to(DEV)
    out, h, c = layer.mixer_prefill(hidden[:, :L].contiguous().to(DEV), wd, pd, pj, **kw, **({"residual": r} if kw else {}))
    ref = P.layer_prefill(x, host, prm, "bf16")
    out_ref, h_ref, c_ref = ref[0], ref[-2], ref[-1]
    assert_close(out, out_ref, TAU, "prefill out", exact_inputs=False)
    if kw:
        assert torch.equal(r.cpu(), want_res)
    for t in range(L, L + steps):
        ht, rt = hidden[:, t].contiguous(), res[:, t].contiguous()
        r = rt.to(DEV)
        more = {}
        x, want_res = reads(ht, rt)
        if kind == "e4m3":
            more = dict(tokens_8bit=True)
            codes, scale = ssm.rms_norm(want_res.to(DEV), norm.to(DEV), eps=EPS, out_dtype=E4M3)
            x = (codes.double() * scale.double()[:, None]).cpu()
        out = layer.mixer_decode_step(ht.to(DEV), wd, pd, pj, h, c, fused=fused, **kw, **({"residual": r} if kw else {}), **more)
        out_ref, _, h_ref, c_ref = P.layer_decode_step(x, host, prm, h_ref, c_ref, "bf16")
        assert_close(out, out_ref, TAU, f"out step {t}", step=t, exact_inputs=False)
        assert_close(h, h_ref, TAU, f"h step {t}", step=t, exact_inputs=False)
        if kw:
            assert torch.equal(r.cpu(), want_res)


HQ, HKV, D, PAGE, DM = 8, 2, 64, 16, 256


def attention(seed=3):
    g = torch.Generator().manual_seed(seed)
    qkv = (torch.randn((HQ + 2 * HKV) * D, DM, generator=g) * DM ** -0.5).bfloat16().to(DEV)
    out = (torch.randn(DM, HQ * D, generator=g) * (HQ * D) ** -0.5).bfloat16().to(DEV)
    return {"qkv": ssm.q4_quantize(qkv), "out": ssm.q4_quantize(out)}


@pytest.mark.parametrize("tokens_8bit", [False, True])
def test_attention_block_on_a_residual_stream(tokens_8bit):
    """The block is the composition of its operators, bit by bit: two prompts, then two decoded tokens."""
    w = attention()
    norm = (1 + 0.1 * torch.randn(DM, generator=torch.Generator().manual_seed(4))).to(DEV)
    freq, ms = ssm.rope_frequencies(D, device=DEV)
    table = torch.tensor([[7, 2, 9], [1, 0, 5]], dtype=torch.int32, device=DEV)
    caches = [ssm.KVCache.allocate(12, PAGE, HKV, D, E4M3, DEV) for _ in range(2)]
    lens = [20, 13]
    cu = torch.tensor([0, 20, 33], dtype=torch.int32, device=DEV)
    seq = torch.cat([torch.full((n,), b) for b, n in enumerate(lens)]).to(DEV)
    pos = torch.cat([torch.arange(n) for n in lens]).to(DEV)

    def by_hand(x, res, cache, attend, positions, slots):
        y = ssm.rms_norm(x, norm, residual=res, eps=EPS, out_dtype=E4M3 if tokens_8bit else None)
        y, scale = y if tokens_8bit else (y, None)
        z = ssm.q4_linear(y, w["qkv"], x_scale=scale).view(len(x), -1, D)
        q, k, v = z[:, :HQ], z[:, HQ:HQ + HKV], z[:, HQ + HKV:]
        kr = torch.empty_like(k)
        q = ssm.kv_write(k, v, cache, slots, q=q, positions=positions, freq=freq, mscale=ms, k_out=kr)
        return ssm.q4_linear(attend(q, kr, v).flatten(1), w["out"])

    x = I.make_hidden(1, 33, DM, "bf16", seed=5)[0].to(DEV)
    res = [torch.randn(33, DM, generator=torch.Generator().manual_seed(6)).to(DEV) for _ in range(2)]
    slots = AL.cache_slots(table, seq, pos, PAGE)
    got = AL.attn_block_prefill(x, w, HQ, caches[0], slots, cu, pos, freq, mscale=ms, norm=norm, residual=res[0], eps=EPS,
                                tokens_8bit=tokens_8bit)
    want = by_hand(x, res[1], caches[1], lambda q, k, v: ssm.attn_prefill(q, k, v, cu), pos, slots)
    assert torch.equal(got, want) and torch.equal(res[0], res[1]) and got.abs().max() > 0
    for step in range(2):
        n = torch.tensor([21 + step, 14 + step], dtype=torch.int32, device=DEV)
        x = I.make_hidden(2, 1, DM, "bf16", seed=7 + step)[:, 0].to(DEV)
        res = [torch.randn(2, DM, generator=torch.Generator().manual_seed(8 + step)).bfloat16().to(DEV) for _ in range(2)]
        p = n.long() - 1
        slots = AL.cache_slots(table, torch.arange(2, device=DEV), p, PAGE)
        got = AL.attn_block_decode(x, w, HQ, caches[0], table, n, freq, mscale=ms, norm=norm, residual=res[0], eps=EPS,
                                   tokens_8bit=tokens_8bit)
        want = by_hand(x, res[1], caches[1], lambda q, k, v: ssm.attn_decode_step(q, caches[1], table, n), p, slots)
        assert torch.equal(got, want) and torch.equal(res[0], res[1])


@pytest.mark.parametrize("rows", [1, 3])
def test_a_captured_decode_step(pj, rows):
    """A decoded token's way through a mixer layer in 4 bits, captured: replays give what eager steps give."""
    w = I.LAYERS["layer_small"]
    prm = I.make_params_distinct(w.d_inner, w.d_state)
    wd, _ = four_bit(I.make_proj_weights(w.d_model, w.d_inner, w.dt_rank, w.d_state, w.io))
    pd = {k: (None if v is None else v.to(DEV)) for k, v in prm.items()}
    norm = torch.ones(w.d_model, device=DEV)
    x = torch.zeros(rows, w.d_model, dtype=torch.bfloat16, device=DEV)
    res = torch.zeros(rows, w.d_model, device=DEV)
    state = [(torch.zeros(rows, w.d_inner, w.d_state, device=DEV), torch.zeros(rows, w.d_inner, 3, device=DEV)) for _ in range(2)]
    bufs = layer.alloc_decode_buffers(x, wd, w.d_state, True, None, True, True)
    kw = dict(fused=True, norm=norm, tokens_8bit=True)

    def run():
        return layer.mixer_decode_step(x, wd, pd, pj, *state[0], residual=res, bufs=bufs, **kw)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        run()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    for t in state[0]:
        t.zero_()
    for t in range(4):
        x.copy_(I.make_hidden(rows, 1, w.d_model, "bf16", seed=20 + t)[:, 0])
        res.fill_(0.1 * t)
        graph.replay()
        torch.cuda.synchronize()
        r = torch.full_like(res, 0.1 * t)
        want = layer.mixer_decode_step(x, wd, pd, pj, *state[1], residual=r, **kw)
        assert torch.equal(out, want) and torch.equal(res, r), t
        assert all(torch.equal(a, b) for a, b in zip(*state)), t


def test_refusals(pj):
    w = I.LAYERS["layer_small"]
    wts = I.make_proj_weights(w.d_model, w.d_inner, w.dt_rank, w.d_state, w.io)
    wd, _ = four_bit(wts)
    plain = {**wd, **{k: wts[k].to(DEV) for k in ("in_xz", "in_x", "in_z")}}
    prm = I.make_params_distinct(w.d_inner, w.d_state)
    pd = {k: (None if v is None else v.to(DEV)) for k, v in prm.items()}
    x = torch.zeros(2, w.d_model, dtype=torch.bfloat16, device=DEV)
    h, c = torch.zeros(2, w.d_inner, w.d_state, device=DEV), torch.zeros(2, w.d_inner, 3, device=DEV)
    norm = torch.ones(w.d_model, device=DEV)
    with pytest.raises(ValueError, match="4 bits"):
        layer.mixer_decode_step(x, plain, pd, pj, h, c, norm=norm, tokens_8bit=True)
    with pytest.raises(ValueError, match="norm"):
        layer.mixer_decode_step(x, wd, pd, pj, h, c, tokens_8bit=True)
    with pytest.raises(ValueError, match="norm"):
        layer.mixer_decode_step(x, wd, pd, pj, h, c, residual=x)
    with pytest.raises(ValueError, match="norm"):
        layer.mixer_prefill(x[:, None], wd, pd, pj, residual=x[:, None])
    with pytest.raises(ValueError, match="norm"):
        B.block_input(x, None, x)
    with pytest.raises(ValueError, match="4 bits"):
        B.project(x.to(E4M3), plain["in_x"], torch.ones(2, device=DEV))
    for a, b in ((0, 8), (8, 32), (16, 16), (0, 10 ** 6)):
        with pytest.raises(ValueError, match="multiples of 16"):
            wd["in_xz"].rows(a, b)
