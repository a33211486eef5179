"""A mixer layer on a stream of its own, while the current stream goes on allocating: what it gives is what it gives alone."""
import pytest
import torch

import selective_state_space_causal_amd as ssm
from selective_state_space_causal_amd import inputs as I
from selective_state_space_causal_amd import layer
from tests.gpu_common import DEV

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pj():
    p = ssm.Projector(DEV)
    yield p
    p.close()


@pytest.mark.parametrize("rows,L", [(1, 40), (2, 37), (1, 2048)])
@pytest.mark.parametrize("fused", [False, True])
def test_mixer_on_a_stream_of_its_own(pj, rows, L, fused):
    w = I.LAYERS["layer_small"]
    wts = {k: v.to(DEV) for k, v in I.make_proj_weights(w.d_model, w.d_inner, w.dt_rank, w.d_state, w.io).items()}
    R, N = wts["x_dt"].shape[0], wts["x_B"].shape[0]
    wts["x_dt"], wts["x_B"], wts["x_C"] = wts["x_all"][:R], wts["x_all"][R:R + N], wts["x_all"][R + N:]
    for k in ("in_xz", "out"):
        wts[k] = ssm.q4_quantize(wts[k])
    wts["in_x"], wts["in_z"] = wts["in_xz"].rows(0, w.d_inner), wts["in_xz"].rows(w.d_inner, 2 * w.d_inner)
    pd = {k: (None if v is None else v.to(DEV)) for k, v in I.make_params_distinct(w.d_inner, w.d_state).items()}
    hidden = I.make_hidden(rows, L + 2, w.d_model, w.io).to(DEV)
    prompt, norm = hidden[:, :L].contiguous(), torch.ones(w.d_model, device=DEV)
    tokens = [hidden[:, L + t].contiguous() for t in range(2)]

    def run(stream):
        """The layer over a prompt and two tokens; on the current stream memory is made and filled after each call."""
        res = torch.zeros_like(prompt, dtype=torch.float32)
        rts = [torch.zeros(rows, w.d_model, device=DEV) for _ in tokens]
        torch.cuda.synchronize()
        if stream is not None:
            with torch.cuda.stream(stream):
                torch.cuda._sleep(20_000_000)  # the layer's work begins once the current stream's memory is filled
        out, h, c = layer.mixer_prefill(prompt, wts, pd, pj, stream=stream, norm=norm, residual=res)
        outs, keep = [out, h, c, res], [fill(prompt)]
        for t, r in zip(tokens, rts):
            outs.append(layer.mixer_decode_step(t, wts, pd, pj, h, c, fused=fused, stream=stream, norm=norm, residual=r, tokens_8bit=True))
            outs.append(r)
            keep.append(fill(t))
        torch.cuda.synchronize()
        assert all(x.isnan().all() for k in keep for x in k)  # and the layer has not written into it
        return outs

    def fill(like):
        sizes = [like.numel(), 2 * rows * w.d_inner * (like.numel() // rows // w.d_model), 2 * w.d_inner * w.d_model,
                 w.d_inner * w.d_model, rows * w.d_inner * N, rows * w.d_model, rows * 2 * w.d_inner, 1024]
        return [torch.full((n,), float("nan"), dtype=dt, device=DEV) for n in sizes for dt in (torch.bfloat16, torch.float32) for _ in range(3)]

    want = run(None)
    for _ in range(2):
        got = run(torch.cuda.Stream())
        for i, (a, b) in enumerate(zip(got, want)):
            assert torch.isfinite(b).all() and torch.equal(a, b), i
