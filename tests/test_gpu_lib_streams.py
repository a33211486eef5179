"""The scan's and the projections' calls on a stream of their own, while the current stream goes on allocating."""
import pytest
import torch

import selective_state_space_causal_amd as ssm
from selective_state_space_causal_amd import inputs as I
from tests.gpu_common import DEV, dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("L", [96, 8192])
def test_calls_on_a_stream_of_their_own(io, L):
    B, D, N, R = 1, 80, 16, 8
    pd = {k: v.to(DEV) for k, v in I.make_params_distinct(D, N).items() if v is not None}
    s = dev(I.make_sequence(B, L, D, N, io))
    w = torch.randn(R + 2 * N, D, device=DEV).to(s["x"].dtype)
    pj = ssm.Projector(DEV)

    def run(stream):
        torch.cuda.synchronize()
        if stream is not None:
            with torch.cuda.stream(stream):
                torch.cuda._sleep(10_000_000)  # the calls' work begins once the current stream's memory is filled
        outs = [*ssm.prefill(s["x"], s["dt"], s["z"], s["Bm"], s["Cm"], pd, stream=stream), ssm.conv_silu(s["x"], pd, stream=stream),
                pj(ssm.PROJ_X, s["x"], w, stream=stream), *ssm.q8_quantize(s["x"], 128, stream=stream)]
        keep = [torch.full((t.numel(),), 7, dtype=t.dtype, device=DEV) for t in outs for _ in range(3)]
        torch.cuda.synchronize()
        assert all((k == 7).all() for k in keep)
        return outs

    want = run(None)
    for a, b in zip(run(torch.cuda.Stream()), want):
        assert torch.equal(a, b)
    pj.close()
