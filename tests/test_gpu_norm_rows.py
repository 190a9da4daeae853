"""The norms' gradients where a block goes through many rows or several wide ones, and rows whose first values
are far from the rest, whose mean takes a second pass.

Bounds and checks are those of test_gpu_norm_grad (a block has at most 4 rows where they are used, and a
column's sum at most 256 blocks). Sums over the rows are exact where rows are of 1 and -1 and gradients small
whole numbers: every partial sum is a whole number under 2^24 in size, which f32 holds in whatever order they
are added, so a row that is left out or taken twice changes the result.
"""
import pytest
import torch

import moe_expert_dispatch_amd as moe
from gpu_common import announce, device
from test_gpu_many_tokens import _free, _need, _repeat, _repeats
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


def _gen(seed):
    return torch.Generator(device=device()).manual_seed(seed)


def _ints(g, most, *shape, dt=F):
    """Whole numbers from -most to most on the generator's device."""
    return torch.randint(-most, most + 1, shape, generator=g, device=g.device, dtype=torch.int8).to(dt)


def _whole(exact):
    assert float(exact.abs().max()) < 2 ** 24
    return exact.to(F)


def _even_rows(g, T, H, dt):
    """Rows of as many 1 as -1 in an order of their own: mean 0 and deviation 1 exactly, so with eps = 0 a
    normalised row is the row itself, whichever way its sums are formed (1 + guess^2 is exact as well)."""
    order = torch.rand(T, H, generator=g, device=g.device).argsort(1)
    return torch.where(order % 2 == 0, 1.0, -1.0).to(dt)


# by the rows that one goes through after the other: a block 59, 16, 3, 4 and 3, a wave 15, half a wave 11;
# then few rows
EVEN = [(60000, 1032), (16384, 2048), (700, 8200), (1000, 16392), (600, 32768), (60000, 264), (170000, 64), (64, 2048),
        (40, 2056), (16, 8192), (2, 8), (1, 520), (2, 1032), (9, 4104), (16, 520), (11, 264)]


@pytest.mark.parametrize("dt", [B, F])
@pytest.mark.parametrize("T,H", EVEN)
def test_norm_sums_over_the_rows(dt, T, H):
    """dgamma = sum of dy n and dbeta = sum of dy, exact."""
    announce(f"exact norm sums {dt} T={T} H={H}")
    g = _gen(T + H)
    x, dy = _even_rows(g, T, H, dt), _ints(g, 2, T, H, dt=dt)
    gamma = torch.ones(H, dtype=dt, device=g.device)
    _, dg, db = moe.layer_norm_backward(dy, x, gamma, 0.0)
    want_g, want_b = (dy * x).double().sum(0), dy.double().sum(0)
    assert torch.equal(dg, _whole(want_g)) and torch.equal(db, _whole(want_b))
    assert torch.equal(moe.rms_norm_backward(dy, x, gamma, 0.0)[1], dg)
    # in place of dy, which the sums have to be formed from first
    dx = dy.clone()
    _, dg2, db2 = moe.layer_norm_backward(dx, x, gamma, 0.0, dx=dx)
    assert torch.equal(dg2, dg) and torch.equal(db2, db)


def test_norm_sums_over_very_many_rows():
    """2^26 rows of 16 values, 4097 of them one after the other in each thread; a period's sums come back 65728 times."""
    dev = device()
    _need(12)
    T, H, period = 2 ** 26 + 7, 16, 1021
    announce(f"exact norm sums T={T}")
    g = _gen(7)
    part, d = _even_rows(g, period, H, B), _ints(g, 1, period, H, dt=B)
    gamma = torch.ones(H, device=dev).bfloat16()
    x, dy = _repeat(part, T), _repeat(d, T)
    whole, rest = T // period, T % period
    total = lambda t: t.double().sum(0) * whole + t[:rest].double().sum(0)  # noqa: E731
    dx, dg, db = moe.layer_norm_backward(dy, x, gamma, 0.0, dx=dy)
    assert _repeats(dx, moe.layer_norm_backward(d, part, gamma, 0.0)[0])
    assert torch.equal(dg, _whole(total(d * part))) and torch.equal(db, _whole(total(d)))
    del x, dy, dx
    _free()
