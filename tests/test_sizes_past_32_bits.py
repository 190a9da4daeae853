"""Sizes that the C ABI's 32-bit integers do not hold are refused by the bindings: ctypes would keep their low
32 bits without a word, so that 2^32 + 8 rows would be 8 rows. No memory is needed: the tensors here are on no
device, and every call has to end before it reaches the library.
"""
import pytest
import torch

import moe_expert_dispatch_amd as moe

ROWS = 2 ** 32 + 8


@pytest.fixture
def unread(monkeypatch):
    """Tensors of the meta device, which hold sizes alone, pass for device tensors; no entry point may be called
    with one."""
    def dev(t, name, dtype=None, shape=None):
        assert shape is None or tuple(t.shape) == tuple(shape), name
        return t

    class NoLib:
        def __getattr__(self, name):
            if name.endswith("_workspace_size"):
                return lambda *a: 16
            raise AssertionError(f"{name} was called")

    monkeypatch.setattr(moe, "_dev", dev)
    monkeypatch.setattr(moe, "_lib", NoLib())
    return lambda *shape, dt=torch.bfloat16: torch.empty(*shape, dtype=dt, device="meta")


def test_the_training_pass(unread):
    t = unread
    x, gamma, off = t(ROWS, 8), t(8), t(3, dt=torch.int32)
    rows, w = t(ROWS, dt=torch.int32), t(ROWS, 1, dt=torch.float32)
    few = t(16, 8)
    for call in (lambda: moe.layer_norm(x, gamma, y=x), lambda: moe.rms_norm(x, gamma, y=x),
                 lambda: moe.layer_norm_backward(x, x, gamma, dx=x), lambda: moe.rms_norm_backward(x, x, gamma, ws=few),
                 lambda: moe.combine_backward(x, x, rows, w, 1), lambda: moe.combine_backward(x, None, rows, None, 1, dy=few),
                 lambda: moe.permute_backward(x, rows, 1), lambda: moe.permute_backward(few, rows, 1),
                 lambda: moe.swiglu(t(ROWS, 16), off), lambda: moe.swiglu(few, t(ROWS, dt=torch.int32)),
                 lambda: moe.grouped_gemm_backward(moe.DOWN, x, off, t(2, 8, 8)),
                 lambda: moe.grouped_gemm_weight_grad(x, x, off), lambda: moe.grouped_gemm_weight_grad(x, x, off, ws=few),
                 lambda: moe.grouped_gemm_weight_grad(t(1, 8), t(1, ROWS), off, ws=few)):
        with pytest.raises(ValueError, match="32 bits"):
            call()


def test_workspace_sizes_and_the_layer():
    for call in (lambda: moe.norm_backward_workspace_size(ROWS, 64), lambda: moe.permute_workspace_size(ROWS, 2, 4),
                 lambda: moe.balance_loss_workspace_size(ROWS, 8, 2), lambda: moe.a2a_dispatch_workspace_size(8, 2, ROWS),
                 lambda: moe.grouped_gemm_weight_grad_workspace_size(torch.bfloat16, 2, ROWS, 64, 64),
                 lambda: moe.ForwardConfig(ROWS, 64, 64, 4, 2, True, 4, torch.bfloat16),
                 lambda: moe.ForwardConfig(4, 64, 64, 4, 2, True, 4, torch.bfloat16, T_max=ROWS)):
        with pytest.raises(ValueError, match="32 bits"):
            call()
    cfg = moe.ForwardConfig(4, 64, 64, 4, 2, True, 4, torch.bfloat16)
    cfg.T = ROWS
    with pytest.raises(ValueError, match="32 bits"):
        moe.forward(cfg, None, None, None)
    assert moe.norm_backward_workspace_size(2 ** 31 - 1, 64) > 0


def test_many_values_in_sizes_that_fit(unread):
    """Tensors of 2^31 values and more, no size of which is: the entry point is called, also one without a size
    among its own arguments."""
    t = unread
    rows = 2 ** 31 // 8 + 1
    x, off = t(rows, 8), t(3, dt=torch.int32)
    cfg = moe.ForwardConfig(rows, 8, 8, 4, 2, True, 4, torch.bfloat16)
    for call in (lambda: moe.forward(cfg, x, t(4, 16, 8), t(4, 8, 8), t(rows, 4, dt=torch.float32)),
                 lambda: moe.layer_norm(x, t(8)), lambda: moe.grouped_gemm_weight_grad(x, x, off)):
        with pytest.raises(AssertionError, match="was called"):
            call()
