"""The norms' gradients where a block goes through several wide rows, and rows whose first values are far
from the rest, whose mean takes a second pass; bounds and checks are those of test_gpu_norm_grad (a block has
at most 4 rows here, and a column's sum at most 256 blocks).
"""
import pytest
import torch

import moe_expert_dispatch_amd as moe
from gpu_common import announce, device
from test_gpu_norm_grad import _check_backward, _check_forward, _inputs

pytestmark = pytest.mark.gpu

B, F = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dt", [B, F])
@pytest.mark.parametrize("T,H", [(600, 8200), (600, 16392), (300, 32768)])
def test_wide_rows_one_after_the_other(dt, T, H):
    dev = device()
    announce(f"norm backward of wide rows {dt} T={T} H={H}")
    x, _, gamma, _, dy, dres = _inputs(T, H, dt, T + H)
    X, G, R = (t.to(dev) for t in (x, gamma, dres))
    for place in ("dy", "x", "dresidual"):
        t = {"dy": dy.to(dev), "x": X.clone(), "dresidual": R.clone()}
        got = moe.layer_norm_backward(t["dy"], t["x"], G, 1e-5, dresidual=t["dresidual"], dx=t[place])
        if place == "dy":
            first = got
            _check_backward(*got, dy, x, gamma, 1e-5, True, dres, "layer")
        assert all(torch.equal(u, v) for u, v in zip(got, first)), place
    D = dy.to(dev)
    dx, dg = moe.rms_norm_backward(D, X, G, 1e-5, dx=D)
    _check_backward(dx, dg, None, dy, x, gamma, 1e-5, False, None, "rms")


@pytest.mark.parametrize("dt", [B, F])
@pytest.mark.parametrize("H", [64, 2056, 4104])
@pytest.mark.parametrize("T", [3, 9, 30, 700])
def test_first_values_far_from_the_rest(dt, H, T):
    """Every other row begins with 8 values 1000 above the others, as a stream with a few large channels does."""
    dev = device()
    announce(f"norm rows of large first values {dt} T={T} H={H}")
    x, _, gamma, beta, dy, dres = _inputs(T, H, dt, 3 * T + H)
    x[::2, :8] = (x[::2, :8].float() + 1000).to(dt)
    X, G, E, D, R = (t.to(dev) for t in (x, gamma, beta, dy, dres))
    y, _, _ = moe.layer_norm(X, G, E, 1e-5)
    _check_forward(y, None, None, x, gamma, beta, 1e-5, None, None, "forward")
    got = moe.layer_norm_backward(D, X, G, 1e-5, dresidual=R)
    _check_backward(*got, dy, x, gamma, 1e-5, True, dres, "layer")
    dx, dg = moe.rms_norm_backward(D, X, G, 1e-5)
    _check_backward(dx, dg, None, dy, x, gamma, 1e-5, False, None, "rms")
