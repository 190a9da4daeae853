"""Gradients of the weighted sum and of the permutation on the GPU against the fp64 oracle.

Tolerances, u = 2^-24: dy is one f32 product and its type's rounding. A dot product of H values passes H / 256 + 16
additions in a thread (8 values of every 256th vector, both vectors of a thread), 6 in the wave, 4 over the
waves: at most H / 256 + 48 roundings of its terms' sum. dx sums K products, K + 2 roundings, and its type's.
"""
import numpy as np
import pytest
import torch

import moe_expert_dispatch_amd as moe
from gpu_common import announce, assert_within, device, np64
from oracle import training as tr

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
ROUND = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
B, F = torch.bfloat16, torch.float32


def _pairs(T, K, g, frac):
    """Rows of the pairs that have one, in an order of their own, with spare rows behind them."""
    P = T * K
    pr = torch.full((P,), -1, dtype=torch.int32)
    has = torch.rand(P, generator=g) < frac
    pr[has] = torch.randperm(int(has.sum()), generator=g).int()
    return pr, int(has.sum())


def _case(T, K, H, seed, frac=0.7):
    g = torch.Generator().manual_seed(seed)
    pr, rows = _pairs(T, K, g, frac)
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    w = torch.rand(T, K, generator=g) * (pr.view(T, K) >= 0)
    return g, pr, rows, w, n(T, H), n(T * K, H), n(T, H)


SHAPES = [(1, 1, 8), (1, 8, 4096), (7, 4, 2048), (33, 3, 520), (5, 32, 72), (9, 9, 1032), (3, 5, 8200), (2, 2, 32768),
          (260, 6, 136), (4, 17, 2056)]


@pytest.mark.parametrize("ddt,ydt", [(B, B), (F, F), (B, F), (F, B)])
@pytest.mark.parametrize("T,K,H", SHAPES)
def test_combine_backward(ddt, ydt, T, K, H):
    dev = device()
    announce(f"combine_backward {ddt} {ydt} T={T} K={K} H={H}")
    _, pr, rows, w, dout, y, _ = _case(T, K, H, T + K + H)
    dout, y = dout.to(ddt), y.to(ydt)
    y[rows:] = float("nan")   # never read
    dy = torch.full((T * K, H), -7.0).to(ydt).to(dev)
    got, dw = moe.combine_backward(dout.to(dev), y.to(dev), pr.to(dev), w.to(dev), K, dy=dy)
    clean = y.clone()
    clean[rows:] = 0
    want, wdw = tr.combine_backward(dout, clean, pr.numpy(), w, K)
    got = np64(got)
    assert (got[rows:] == -7).all()
    assert_within(got[:rows], want[:rows], (ROUND[ydt] + 2 * U) * np.abs(want[:rows]) + 1e-44, "dy")
    size = np.abs(tr.combine_backward(dout.abs(), clean.abs(), pr.numpy(), w, K)[1])
    assert_within(np64(dw), wdw, (H / 256 + 48) * U * size + 1e-44, "dw")
    assert (np64(dw).reshape(-1)[pr.numpy() < 0] == 0).all()
    # without weights: dout's rows themselves, and y need not be there
    got, none = moe.combine_backward(dout.to(dev), None, pr.to(dev), None, K, dy=dy)
    assert none is None
    for p, r in enumerate(pr.tolist()):
        if r >= 0:
            assert torch.equal(got[r].cpu(), dout[p // K].to(ydt)), p


@pytest.mark.parametrize("dt,xdt", [(B, B), (F, F), (B, F), (F, B)])
@pytest.mark.parametrize("T,K,H", SHAPES)
def test_permute_backward(dt, xdt, T, K, H):
    dev = device()
    announce(f"permute_backward {dt} {xdt} T={T} K={K} H={H}")
    g, pr, rows, w, x, dxp, before = _case(T, K, H, 3 * T + K + H)
    x, dxp, before = x.to(dt), dxp.to(dt), before.to(xdt)
    dxp[rows:] = float("nan")
    clean = dxp.clone()
    clean[rows:] = 0
    X, D, P, W = x.to(dev), dxp.to(dev), pr.to(dev), w.to(dev)
    for ww in (w, None):
        want, wdw = tr.permute_backward(clean, pr.numpy(), K, ww, x)
        size = tr.permute_backward(clean.abs(), pr.numpy(), K, ww, x.abs())
        allow = (K + 2) * U * size[0]
        for acc in (False, True):
            dx = before.to(dev) if acc else None
            if ww is None:
                got, dw = moe.permute_backward(D, P, K, dx=dx, dx_dtype=xdt, accumulate=acc)
                assert dw is None
            else:
                got, dw = moe.permute_backward(D, P, K, W, X, dx=dx, dx_dtype=xdt, accumulate=acc)
                assert_within(np64(dw), wdw, (H / 256 + 48) * U * size[1] + 1e-44, "dpair_w")
                only, none = moe.permute_backward(D, P, K, W, dx=before.to(dev) if acc else None, dx_dtype=xdt,
                                                  accumulate=acc)
                assert none is None and torch.equal(only, got)
            ref = want + (np64(before) if acc else 0)
            err = allow + U * np.abs(ref)
            assert_within(np64(got), ref, err + ROUND[xdt] * (np.abs(ref) + err) + 1e-44, f"dx acc {acc}")


def test_no_pairs_no_tokens():
    dev = device()
    pr = torch.full((6,), -1, dtype=torch.int32, device=dev)
    d, y = torch.randn(3, 64, device=dev), torch.empty(0, 64, device=dev)
    dy, dw = moe.combine_backward(d, y, pr, torch.ones(3, 2, device=dev), 2)
    assert dy.shape == (0, 64) and not dw.any()
    dx, dpw = moe.permute_backward(torch.randn(6, 64, device=dev), pr, 2, torch.ones(3, 2, device=dev), d)
    assert not dx.any() and not dpw.any()
    none = torch.empty(0, 64, device=dev)
    dy, dw = moe.combine_backward(none, y, pr[:0], torch.ones(0, 2, device=dev), 2)
    assert dw.shape == (0, 2)
    assert moe.permute_backward(y, pr[:0], 2)[0].shape == (0, 64)


def test_values_behind_pairs_without_a_row():
    """A pair without a row gives no gradient, whatever its weight and its token hold."""
    dev = device()
    T, K, H = 5, 4, 264
    g, pr, rows, w, dout, y, x = _case(T, K, H, 9, 0.5)
    w[pr.view(T, K) < 0] = float("nan")
    dy, dw = moe.combine_backward(dout.to(dev), y.to(dev), pr.to(dev), w.to(dev), K)
    dx, dpw = moe.permute_backward(y.to(dev), pr.to(dev), K, w.to(dev), x.to(dev))
    for t in (dw, dx, dpw, dy[:rows]):
        assert torch.isfinite(t).all()
    out = (pr.view(T, K) < 0)
    assert not dw.cpu()[out].any() and not dpw.cpu()[out].any()


def test_runs_repeat_bit_for_bit():
    dev = device()
    _, pr, _, w, dout, y, x = (t.to(dev) if isinstance(t, torch.Tensor) else t for t in _case(500, 8, 1032, 4, 0.9))
    first = moe.combine_backward(dout, y, pr, w, 8, dy=torch.zeros_like(y)) + moe.permute_backward(y, pr, 8, w, x)
    for _ in range(3):
        again = moe.combine_backward(dout, y, pr, w, 8, dy=torch.zeros_like(y)) + moe.permute_backward(y, pr, 8, w, x)
        assert all(torch.equal(u, v) for u, v in zip(first, again))


def test_refusals():
    dev = device()
    _, pr, _, w, dout, y, x = (t.to(dev) if isinstance(t, torch.Tensor) else t for t in _case(4, 2, 64, 1))
    for bad in (lambda: moe.combine_backward(dout, y, pr.long(), w, 2), lambda: moe.combine_backward(dout.half(), y, pr, w, 2),
                lambda: moe.combine_backward(dout, y, pr, w.double(), 2),
                lambda: moe.permute_backward(y, pr, 2, w, x.bfloat16())):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: moe.combine_backward(dout, y, pr, w, 3), lambda: moe.combine_backward(dout[:3], y, pr, w, 2),
                lambda: moe.combine_backward(dout, y[:, :32], pr, w, 2), lambda: moe.combine_backward(dout, None, pr, None, 2),
                lambda: moe.combine_backward(dout, None, pr, w, 2, dy=y), lambda: moe.combine_backward(dout, y, pr, w[:3], 2),
                lambda: moe.combine_backward(dout, y, pr, None, 2, dw=w), lambda: moe.permute_backward(y, pr, 2, x=x),
                lambda: moe.permute_backward(y, pr, 2, accumulate=True), lambda: moe.permute_backward(y, pr, 2, w, dpair_w=w),
                lambda: moe.permute_backward(y, pr.cpu(), 2)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(RuntimeError):
        moe.combine_backward(dout, y, pr, w, 2, dy=y)
    with pytest.raises(RuntimeError):
        moe.permute_backward(y, pr, 2, w, x, dx=x)
