"""The conv front's calls read x as a contiguous [B, D, L] tensor, so another is refused (no GPU: host tensors that say they are on
one, and a library that launches nothing)."""
import pytest
import torch

from selective_state_space_causal_amd import _lib as L

B, D, S, R, N = 2, 16, 8, 4, 16


class OnGpu(torch.Tensor):
    is_cuda = property(lambda self: True)
    device = property(lambda self: torch.device("cuda:0"))

    def get_device(self):
        return 0


class Library:
    def __getattr__(self, name):
        return lambda *a: 0


def gpu(t):
    return t.as_subclass(OnGpu)


@pytest.mark.parametrize("x,fits", [(torch.zeros(B, D, S), True), (torch.zeros(B, D, 2 * S)[..., :S], False),
                                    (torch.zeros(B, S, D).transpose(1, 2), False)])
def test_x_is_contiguous(monkeypatch, x, fits):
    monkeypatch.setattr(L, "load", Library)
    monkeypatch.setattr(L, "stream_handle", lambda s, d=None: 0)
    params, w = {"conv_w": gpu(torch.zeros(D, 4))}, gpu(torch.zeros(R + 2 * N, D))
    outs = dict(lowrank=gpu(torch.zeros(B, S, R)), Bm=gpu(torch.zeros(B, S, N)), Cm=gpu(torch.zeros(B, S, N)))
    for call in (lambda: L.conv_silu(gpu(x), params, u=gpu(torch.zeros(B, D, S))), lambda: L.conv_xproj(gpu(x), params, w, R, **outs)):
        if fits:
            call()
        else:
            with pytest.raises(ValueError, match="x must be a contiguous"):
                call()
