"""The training pass past 32 bits: rows whose launches pass the 2^32 threads of one grid dimension, and buffers
of more than 2^31 values. Inputs repeat after a short period, and so have the outputs to, or a few rows are
checked against the fp64 oracle.
"""
import pytest
import torch

import moe_expert_dispatch_amd as moe
from gpu_common import announce, assert_within, device, np64
from oracle import training as tr
from test_gpu_many_tokens import _free, _need, _repeat, _repeats

pytestmark = pytest.mark.gpu

PERIOD = 1021
U = 2.0 ** -24


def test_layer_norm_rows():
    dev = device()
    _need(12)
    for T, H in ((2 ** 28 + 7, 8), (2 ** 26 + 7, 24)):   # rows of 16 lanes, 16 to a block of 256 threads
        announce(f"layer_norm T={T} H={H}")
        g = torch.Generator().manual_seed(1)
        part, gamma = torch.randn(PERIOD, H, generator=g).bfloat16().to(dev), torch.ones(H).bfloat16().to(dev)
        x = _repeat(part, T)
        y, _, _ = moe.layer_norm(x, gamma, gamma, 1e-5, y=x)
        assert _repeats(y, moe.layer_norm(part, gamma, gamma, 1e-5)[0])
        del x, y
        _free()


def test_norm_backward_rows():
    """dgamma and dbeta are sums of 2^26 equal rows' terms in chains of 2^16 and more: 2^-8 of their size."""
    dev = device()
    _need(12)
    T, H = 2 ** 26 + 7, 16
    announce(f"norm backward T={T}")
    g = torch.Generator().manual_seed(2)
    part, d = (torch.randn(PERIOD, H, generator=g).bfloat16().to(dev) for _ in range(2))
    gamma = torch.ones(H).bfloat16().to(dev)
    x, dy = _repeat(part, T), _repeat(d, T)
    dx, dg, db = moe.layer_norm_backward(dy, x, gamma, 1e-5, dx=dy)
    assert _repeats(dx, moe.layer_norm_backward(d, part, gamma, 1e-5)[0])
    n, _ = tr.normalise(part, 1e-5, True)
    times = T / PERIOD
    size = abs(np64(d) * n).sum(0) * times
    assert_within(np64(dg), (np64(d) * n).sum(0) * times, 2.0 ** -8 * size, "dgamma")
    assert_within(np64(db), np64(d).sum(0) * times, 2.0 ** -8 * abs(np64(d)).sum(0) * times, "dbeta")
    del x, dy, dx
    _free()


def test_dispatch_rows():
    """A wave a token: 2^32 threads at 2^26 tokens."""
    dev = device()
    _need(12)
    T, H = 2 ** 26 + 7, 8
    announce(f"dispatch gradients T={T}")
    g = torch.Generator().manual_seed(3)
    n = lambda *s: torch.randn(*s, generator=g).bfloat16().to(dev)  # noqa: E731
    pd, py, px = n(PERIOD, H), n(PERIOD, H), n(PERIOD, H)
    pw = torch.rand(PERIOD, 1, generator=g).to(dev)
    rows = torch.arange(T, dtype=torch.int32, device=dev)
    short = rows[:PERIOD].contiguous()
    d, y, w = _repeat(pd, T), _repeat(py, T), _repeat(pw, T)
    dy, dw = moe.combine_backward(d, y, rows, w, 1)
    sy, sw = moe.combine_backward(pd, py, short, pw, 1)
    assert _repeats(dy, sy) and _repeats(dw, sw)
    del dy, dw, d
    _free()
    x = _repeat(px, T)
    dx, dpw = moe.permute_backward(y, rows, 1, w, x)
    sx, spw = moe.permute_backward(py, short, 1, pw, px)
    assert _repeats(dx, sx) and _repeats(dpw, spw)
    del dx, dpw, x, y, w, rows
    _free()


def test_swiglu_past_31_bits():
    dev = device()
    _need(20)
    rows, I = 2 ** 19 + 5, 2048   # h of 2^31 values and more
    announce(f"swiglu rows={rows} I={I}")
    part = torch.randn(PERIOD, 2 * I, generator=torch.Generator().manual_seed(4)).bfloat16().to(dev)
    off = torch.tensor([0, 5, rows], dtype=torch.int32, device=dev)
    act = moe.swiglu(_repeat(part, rows), off)
    assert _repeats(act, moe.swiglu(part, torch.tensor([0, PERIOD], dtype=torch.int32, device=dev)))
    del act
    _free()


@pytest.mark.parametrize("dt,rows,wide", [(torch.bfloat16, 70001, 32768), (torch.float32, 70001, 32768)])
def test_products_past_31_bits(dt, rows, wide):
    """Rows that lie past 2^31 values of their buffer, as output of the rows' gradient and as its and the
    weights' gradient's input."""
    dev = device()
    _need(40)
    announce(f"gradients of {rows} rows of {wide} {dt}")
    g = torch.Generator().manual_seed(5)
    n = lambda *s: torch.randn(*s, generator=g).to(dt).to(dev)  # noqa: E731
    off = torch.tensor([0, 100, 100, rows], dtype=torch.int32, device=dev)
    dc, w = n(rows, 16), n(3, 16, wide)
    out = moe.grouped_gemm_backward(moe.DOWN, dc, off, w)
    at = torch.tensor([0, 99, 100, 101, 65536, 65537, rows - 1], device=dev)
    slot = torch.tensor([0, 0, 2, 2, 2, 2, 2], device=dev)
    rnd = 2.0 ** -8 if dt == torch.bfloat16 else U
    for r, s in zip(at.tolist(), slot.tolist()):
        want = np64(dc[r]) @ np64(w[s])
        size = abs(np64(dc[r])) @ abs(np64(w[s]))
        assert_within(np64(out[r]), want, 33 * U * size + rnd * (abs(want) + 33 * U * size) + 1e-40, f"row {r}")
    # out as dc of the other two: a whole row contracted, and the rows of a slot
    back = n(3, wide, 8)
    got = moe.grouped_gemm_backward(moe.DOWN, out, off, back)
    for r, s in zip(at.tolist(), slot.tolist()):
        want, size = np64(out[r]) @ np64(back[s]), abs(np64(out[r])) @ abs(np64(back[s]))
        assert_within(np64(got[r]), want, 2 * wide * U * size + rnd * (abs(want) + size) + 1e-40, f"row {r} back")
    a = n(rows, 8)
    dw = moe.grouped_gemm_weight_grad(out, a, off)
    assert not dw[1].any()
    cols = torch.tensor([0, 1, 255, 256, 32760, 32767], device=dev)
    for s, lo, hi in ((0, 0, 100), (2, 100, rows)):
        c, b = np64(out[lo:hi][:, cols]), np64(a[lo:hi])
        assert_within(np64(dw[s, cols]), c.T @ b, 2 * rows * U * (abs(c).T @ abs(b)) + 1e-40, f"slot {s}")
    del out, dw, got
    _free()
