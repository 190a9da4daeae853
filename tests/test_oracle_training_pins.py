"""The training pass's fp64 formulas against central differences of the values they are gradients of.

A central difference with step e is off by e^2 / 6 times a third derivative and 2^-53 / e of the value: with
e = 1e-5 and values and derivatives of order 1 to 100, under 1e-7.
"""
import numpy as np
import pytest

from oracle import training as tr

STEP, TOL = 1e-5, 1e-6


def _difference(f, x, at):
    a, b = x.copy(), x.copy()
    a[at] += STEP
    b[at] -= STEP
    return (f(a) - f(b)) / (2 * STEP)


def _check(f, x, grad, rng, n=12):
    for _ in range(n):
        at = tuple(int(rng.integers(0, s)) for s in x.shape)
        d = _difference(f, x, at)
        assert abs(d - grad[at]) <= TOL * (1 + abs(d)), (at, d, grad[at])


@pytest.mark.parametrize("centred", [True, False])
def test_norm(centred):
    rng = np.random.default_rng(1)
    x, dy, res = (rng.standard_normal((3, 16)) for _ in range(3))
    gamma, beta = rng.standard_normal(16), rng.standard_normal(16)

    def value(x, gamma, beta):
        n, _ = tr.normalise(x, 1e-3, centred)
        return (dy * (n * gamma + (beta if centred else 0))).sum() + (res * x).sum()

    dx, dg, db = tr.norm_backward(dy, x, gamma, 1e-3, centred, res)
    _check(lambda v: value(v, gamma, beta), x, dx, rng)
    _check(lambda v: value(x, v, beta), gamma, dg, rng)
    if centred:
        _check(lambda v: value(x, gamma, v), beta, db, rng)
        _, v = tr.layer_norm(x, gamma, beta, 1e-3)
        assert np.allclose((v - beta) / gamma, tr.normalise(x, 1e-3, True)[0], rtol=1e-12)


def test_combine_and_permute():
    rng = np.random.default_rng(2)
    T, K, H, rows = 4, 3, 8, 10
    pr = rng.permutation(rows)[:rows].tolist() + [-1] * (T * K - rows)
    pr = rng.permutation(np.array(pr))
    y, w, dout = rng.standard_normal((rows, H)), rng.random((T, K)), rng.standard_normal((T, H))

    def combined(y, w):
        return sum((dout[p // K] * w[p // K, p % K] * y[r]).sum() for p, r in enumerate(pr) if r >= 0)

    dy, dw = tr.combine_backward(dout, y, pr, w, K)
    _check(lambda v: combined(v, w), y, dy, rng)
    _check(lambda v: combined(y, v), w, dw, rng)
    assert (dw.reshape(-1)[pr < 0] == 0).all()
    x, dxp = rng.standard_normal((T, H)), rng.standard_normal((rows, H))

    def permuted(x, w):
        return sum((dxp[r] * w[p // K, p % K] * x[p // K]).sum() for p, r in enumerate(pr) if r >= 0)

    dx, dpw = tr.permute_backward(dxp, pr, K, w, x)
    _check(lambda v: permuted(v, w), x, dx, rng)
    _check(lambda v: permuted(x, v), w, dpw, rng)


def test_experts():
    rng = np.random.default_rng(3)
    S, H, I, off = 3, 8, 6, [0, 4, 4, 9]
    x, dy = rng.standard_normal((9, H)), rng.standard_normal((9, H))
    wg, wd = rng.standard_normal((S, 2 * I, H)), rng.standard_normal((S, H, I))

    def rows(a, w):  # the grouped product itself
        return np.concatenate([a[off[s]:off[s + 1]] @ w[s].T for s in range(S)])

    def value(x, wg, wd):
        return (dy * rows(tr.swiglu(rows(x, wg)), wd)).sum()

    h = rows(x, wg)
    act = tr.swiglu(h)
    dh = tr.swiglu_backward(h, tr.grouped_rows_grad(dy, off, wd))
    _check(lambda v: value(v, wg, wd), x, tr.grouped_rows_grad(dh, off, wg), rng)
    _check(lambda v: value(x, v, wd), wg, tr.grouped_weight_grad(dh, x, off), rng)
    _check(lambda v: value(x, wg, v), wd, tr.grouped_weight_grad(dy, act, off), rng)
    assert not tr.grouped_weight_grad(dy, act, off)[1].any()
