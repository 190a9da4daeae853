"""The SwiGLU and its gradient over the whole range of the gate.

A sigmoid under 2^-126, f32's least normal number (a gate under -87.3), may count as 0: its product with g u is
then off by |g u| 2^-126 at most, and s (1 + g (1 - s)) by (1 + |g|) 2^-126. Everywhere else the bounds of
test_gpu_experts_grad hold: 4 u (|g| + 6) relative for the sigmoid's products, 8 u (|g| + 6) (1 + |g|) s for the
gradient's factor, u = 2^-24, and the output's rounding.
"""
import numpy as np
import pytest
import torch

import moe_expert_dispatch_amd as moe
from gpu_common import announce, assert_within, device, np64
from oracle import training as tr

pytestmark = pytest.mark.gpu

U, LEAST = 2.0 ** -24, 2.0 ** -126
ROUND = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
TINY = 1e-40
GATES = [0.0, -0.0, 1.0, -1.0, 16.0, -16.0, 60.0, -60.0, 86.0, -86.0, -87.0, -87.5, -88.0, -88.5, -89.0, -90.0, -103.0, -104.0,
         -110.0, -200.0, 88.0, 89.0, 104.0, 200.0, 1e10, -1e10, 1e30, -1e30, 1e-30, -1e-30, 3e-39, -3e-39]


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_gates_of_every_size(dt):
    dev = device()
    announce(f"swiglu over the gate's range {dt}")
    ups = [1.0, -0.75, 1e-8, 2.0 ** 20, -1e7]
    I, rows = len(GATES), len(ups)
    h = torch.cat([torch.tensor(GATES).expand(rows, I), torch.tensor(ups)[:, None].expand(rows, I)], 1).to(dt)
    off = torch.tensor([0, rows], dtype=torch.int32, device=dev)
    hd = np64(h)
    g, u = hd[:, :I], hd[:, I:]
    s = tr.sigmoid(g)
    act = moe.swiglu(h.to(dev), off)
    want = g * s * u
    err = 4 * U * (np.abs(g) + 6) * np.abs(want) + LEAST * np.abs(g * u)
    assert_within(np64(act), want, err + ROUND[dt] * (np.abs(want) + err) + TINY, "act")
    gen = torch.Generator().manual_seed(1)
    dy, w = torch.randn(rows, 16, generator=gen).to(dt), torch.randn(1, 16, I, generator=gen).to(dt)
    dh = moe.grouped_gemm_backward(moe.DOWN, dy.to(dev), off, w.to(dev), h=h.to(dev))
    da, size = np64(dy) @ np64(w)[0], np.abs(np64(dy)) @ np.abs(np64(w)[0])
    f, e = s * (1 + g * (1 - s)), 8 * U * (np.abs(g) + 6) * s * (1 + np.abs(g)) + LEAST * (1 + np.abs(g))
    for got, part, slope, wide in ((dh[:, :I], da * u * f, np.abs(u * f), np.abs(u) * e),
                                   (dh[:, I:], da * g * s, np.abs(g * s), 8 * U * (np.abs(g) + 6) * np.abs(g * s) + LEAST * np.abs(g))):
        err = 33 * U * size * (slope + wide) + np.abs(da) * wide
        assert_within(np64(got), part, err + ROUND[dt] * (np.abs(part) + err) + TINY, "dh")
