"""A workspace that holds one byte over and over (or every other one) has the bytes that are asked for, but not the
memory: refused by every call that takes one, before any launch. Seen without a device, on tensors of the
meta device.
"""
import pytest
import torch

import moe_expert_dispatch_amd as moe

B, F, I32, U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8


def _t(*shape, dt=B):
    return torch.empty(*shape, dtype=dt, device="meta")


@pytest.fixture
def no_launch(monkeypatch):
    def dev(t, name, dtype=None, shape=None):
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        return t

    def launch(what, *rest):
        raise AssertionError(f"{what} was launched")

    monkeypatch.setattr(moe, "_dev", dev)
    monkeypatch.setattr(moe, "_launch", launch)
    monkeypatch.setattr(moe, "_lib", type("Sizes", (), {"__getattr__": lambda self, name: (lambda *a: 16)})())


CALLS = {
    "permute": lambda ws: moe.permute(_t(6, 16), _t(6, 2, dt=I32), _t(6, 2, dt=U8), 4, ws=ws),
    "balance_loss": lambda ws: moe.balance_loss(_t(6, 8, dt=F), _t(6, 2, dt=I32), 0.1, ws=ws),
    "forward": lambda ws: moe.forward(moe.ForwardConfig(6, 16, 8, 4, 2, True, 4, B), _t(6, 16), _t(4, 16, 16), _t(4, 16, 8),
                                      _t(6, 4, dt=F), ws=ws),
    "a2a_dispatch": lambda ws: moe.a2a_dispatch(_t(6, 16), _t(6, 2, dt=I32), _t(6, 2, dt=F), 4, 2, ws=ws),
    "layer_norm_backward": lambda ws: moe.layer_norm_backward(_t(6, 16), _t(6, 16), _t(16), ws=ws),
    "rms_norm_backward": lambda ws: moe.rms_norm_backward(_t(6, 16), _t(6, 16), _t(16), ws=ws),
    "grouped_gemm_weight_grad": lambda ws: moe.grouped_gemm_weight_grad(_t(6, 16), _t(6, 8), _t(3, dt=I32), ws=ws),
}


@pytest.mark.parametrize("what", list(CALLS))
def test_a_workspace_is_contiguous(no_launch, what):
    for ws in (_t(1, dt=U8).expand(1 << 24), _t(1 << 24, dt=U8)[::2]):
        with pytest.raises(ValueError, match="ws must be contiguous"):
            CALLS[what](ws)
    with pytest.raises(AssertionError, match="launched"):
        CALLS[what](_t(1 << 24, dt=U8))
