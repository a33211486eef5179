"""A refused call on a residual stream, put right and made again, adds hidden once."""
import pytest
import torch

import selective_state_space_causal_amd as ssm
from selective_state_space_causal_amd import attn_layer as AL
from selective_state_space_causal_amd import inputs as I
from selective_state_space_causal_amd import layer
from tests.gpu_common import DEV

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pj():
    p = ssm.Projector(DEV)
    yield p
    p.close()


def again(call, good, wrong, res, hidden):
    """call(good with one of wrong's) raises and leaves res; call(good) adds hidden."""
    before = res.clone()
    for kw in wrong:
        with pytest.raises((ValueError, TypeError, KeyError, ssm.SsmError)):
            call({**good, **kw})
        torch.cuda.synchronize()
        assert torch.equal(res, before), sorted(kw)
    out = call(good)
    assert torch.equal(res, before + hidden.float()) and torch.isfinite(out).all()


@pytest.mark.parametrize("rows", [1, 2])
@pytest.mark.parametrize("q4", [False, True])
@pytest.mark.parametrize("kind", ["prefill", "fused", "unfused"])
def test_mixer(pj, rows, q4, kind):
    w = I.LAYERS["layer_small"]
    wd = {k: v.to(DEV) for k, v in I.make_proj_weights(w.d_model, w.d_inner, w.dt_rank, w.d_state, w.io).items()}
    R, N = wd["x_dt"].shape[0], wd["x_B"].shape[0]
    wd["x_dt"], wd["x_B"], wd["x_C"] = wd["x_all"][:R], wd["x_all"][R:R + N], wd["x_all"][R + N:]
    if q4:
        for k in ("in_xz", "out"):
            wd[k] = ssm.q4_quantize(wd[k])
        wd["in_x"], wd["in_z"] = wd["in_xz"].rows(0, w.d_inner), wd["in_xz"].rows(w.d_inner, 2 * w.d_inner)
    pd = {k: (None if v is None else v.to(DEV)) for k, v in I.make_params_distinct(w.d_inner, w.d_state).items()}
    L = 16
    hidden = I.make_hidden(rows, L, w.d_model, w.io).to(DEV)
    if kind != "prefill":
        hidden = hidden[:, 0].contiguous()
    res, norm = torch.randn(hidden.shape, device=DEV), torch.ones(w.d_model, device=DEV)
    good = dict(w=wd, p=pd, h=torch.zeros(rows, w.d_inner, w.d_state, device=DEV), c=torch.zeros(rows, w.d_inner, 3, device=DEV))

    def call(a):
        if kind == "prefill":
            return layer.mixer_prefill(hidden, a["w"], a["p"], pj, norm=norm, residual=res)[0]
        return layer.mixer_decode_step(hidden, a["w"], a["p"], pj, a["h"], a["c"], fused=kind == "fused", norm=norm, residual=res)
    wrong = [dict(w=dict(wd, dt=wd["dt"][:, :-1])), dict(w=dict(wd, out=torch.zeros(w.d_model, 32, dtype=torch.bfloat16, device=DEV))),
             dict(w={k: v for k, v in wd.items() if k != "out"}), dict(p=dict(pd, conv_w=pd["conv_w"].cpu())), dict(p=dict(pd, A=pd["A"][:-1]))]
    if kind != "prefill":
        wrong += [dict(h=good["h"][:, :-1]), dict(c=good["c"].bfloat16())]
    again(call, good, wrong, res, hidden)


@pytest.mark.parametrize("q4", [False, True])
@pytest.mark.parametrize("decode", [False, True])
def test_attention_block(q4, decode):
    Hq, Hkv, D, page, DM, T = 4, 2, 64, 16, 128, 3
    w = {"qkv": torch.randn((Hq + 2 * Hkv) * D, DM, device=DEV).bfloat16() / 8, "out": torch.randn(DM, Hq * D, device=DEV).bfloat16() / 8}
    if q4:
        w = {k: ssm.q4_quantize(v) for k, v in w.items()}
    freq, ms = ssm.rope_frequencies(D, device=DEV)
    cache = ssm.KVCache.allocate(8, page, Hkv, D, torch.float8_e4m3fn, DEV)
    for t in (cache.k, cache.v):
        t.view(torch.uint8).zero_()
    cache.k_scale.zero_(), cache.v_scale.zero_()
    hidden, norm = torch.randn(T, DM, device=DEV).bfloat16(), torch.ones(DM, device=DEV)
    res, i32 = torch.randn(T, DM, device=DEV), dict(dtype=torch.int32, device=DEV)
    good = dict(w=w, slots=torch.arange(T, device=DEV), cu=torch.tensor([0, T], **i32), pos=torch.arange(T, device=DEV), freq=freq,
                table=torch.arange(T, **i32)[:, None].contiguous(), lens=torch.ones(T, **i32))

    def call(a):
        if decode:
            return AL.attn_block_decode(hidden, a["w"], Hq, cache, a["table"], a["lens"], a["freq"], mscale=ms, norm=norm, residual=res)
        return AL.attn_block_prefill(hidden, a["w"], Hq, cache, a["slots"], a["cu"], a["pos"], a["freq"], mscale=ms, norm=norm, residual=res)
    wrong = [dict(w=dict(w, out=torch.zeros(DM, Hq * D - 16, dtype=torch.bfloat16, device=DEV))), dict(w={"qkv": w["qkv"]}),
             dict(freq=freq.float())]
    wrong += [dict(table=good["table"].long()), dict(lens=good["lens"][:-1])] if decode else \
        [dict(slots=good["slots"].int()), dict(pos=good["pos"][:-1]), dict(cu=good["cu"].long())]
    again(call, good, wrong, res, hidden)
