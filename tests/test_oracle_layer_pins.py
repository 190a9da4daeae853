"""Pins of the oracles of the norm, the router's loss and gradient, and the
MXFP4 weights: closed forms, hand-derived vectors, autograd and differences.
"""
import numpy as np
import pytest
import torch

import oracle


def test_rms_norm_closed_forms():
    x = np.array([[3.0, -4.0], [0.0, 0.0]])
    h, v = oracle.rms_norm(x, np.array([1.0, 2.0]), 0.0 + 12.5)
    assert np.array_equal(h, x)
    # mean(h^2) = 12.5, so the first row is divided by 5
    assert np.allclose(v, [[0.6, -1.6], [0.0, 0.0]], rtol=1e-15)
    h, _ = oracle.rms_norm(x, np.ones(2), 1.0, residual=np.ones((2, 2)))
    assert np.array_equal(h, x + 1)


def test_balance_loss_of_even_and_collapsed_routing():
    # every expert equally likely and equally loaded: coef exactly
    T, E, K = 8, 4, 2
    ids = np.array([[t % 4, (t + 1) % 4] for t in range(T)])
    loss, counts, prob = oracle.balance_loss(np.zeros((T, E)), ids, 0.5)
    assert loss == 0.5 and list(counts) == [4, 4, 4, 4, 8] and np.array_equal(prob, np.full(E, 0.25))
    # everything to one expert with probability 1: coef * E / K
    l = np.full((T, E), -1e9)
    l[:, 2] = 0
    loss, counts, _ = oracle.balance_loss(l, np.full((T, 1), 2), 1.0)
    assert loss == E and counts[2] == T
    # masked tokens have no influence; nothing valid gives zeros
    l[3] = np.nan
    m = np.ones(T)
    m[3] = 0
    assert oracle.balance_loss(l, np.full((T, 1), 2), 1.0, m)[0] == E
    assert oracle.balance_loss(l, np.full((T, 1), 2), 1.0, np.zeros(T))[0] == 0.0


@pytest.mark.parametrize("renorm", [False, True])
def test_route_backward_is_autograd_and_differences(renorm):
    g = torch.Generator().manual_seed(3)
    T, E, K, coef, dloss = 6, 9, 3, 0.7, 1.3
    l = torch.randn(T, E, generator=g, dtype=torch.float64, requires_grad=True)
    ids = torch.stack([torch.randperm(E, generator=g)[:K] for _ in range(T)])
    dw = torch.randn(T, K, generator=g, dtype=torch.float64)
    mask = torch.tensor([1, 1, 0, 1, 1, 1])
    _, counts, _ = oracle.balance_loss(l.detach(), ids, coef, mask)
    got = oracle.route_backward(l.detach(), ids, dw, renorm, counts, coef, dloss, mask)

    ok = mask.bool()
    p = torch.softmax(l[ok], 1)
    w = p.gather(1, ids[ok])
    w = w / w.sum(1, keepdim=True) if renorm else w
    n = int(ok.sum())
    f = torch.from_numpy(counts[:E] / (n * K))
    ((w * dw[ok]).sum() + dloss * coef * E * (f * p.mean(0)).sum()).backward()
    assert np.allclose(got, l.grad.numpy(), rtol=1e-12, atol=1e-15)
    assert not got[2].any()

    def value(x):  # the counts stay as they are: the gradient takes them as constants
        w = oracle.routing_weights(x, ids, renorm)[ok.numpy()]
        return (w * dw.numpy()[ok]).sum() + dloss * oracle.balance_loss(x, ids, coef, mask, counts)[0]
    base, h = l.detach().numpy(), 1e-6
    for t, e in [(0, 0), (1, int(ids[1, 0])), (5, 8)]:
        up, down = base.copy(), base.copy()
        up[t, e] += h
        down[t, e] -= h
        # central difference: truncation h^2/6 times a third derivative of order 1, rounding 1e-16/h
        assert abs((value(up) - value(down)) / (2 * h) - got[t, e]) < 1e-8


def test_route_backward_repeated_and_foreign_ids():
    l = np.log(np.array([[0.5, 0.25, 0.25]]))
    # the same expert twice: its two upstream values add
    a = oracle.route_backward(l, np.array([[1, 1]]), np.array([[2.0, 3.0]]), False)
    b = oracle.route_backward(l, np.array([[1, -1]]), np.array([[5.0, 99.0]]), False)
    assert np.allclose(a, b, rtol=1e-15)
    assert np.allclose(b, [[-0.625, 0.25 * 5 * 0.75, -0.3125]], rtol=1e-12)


def test_mxfp4_by_hand():
    w = np.zeros(32)
    w[:10] = [6.0, -0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.9, -0.0]
    codes, b = oracle.mxfp4_encode(w)
    assert b[0] == 127  # amax 7.9: floor(log2) = 2, 2^(2-2) = 1
    # ties to the even code: .25 -> 0, .75 -> 1, 1.25 -> 1, 1.75 -> 2, 2.5 -> 2, 3.5 -> 4, 5 -> 4
    assert list(oracle.mxfp4_decode(codes, b)[:10]) == [6, 0, 1, 1, 2, 2, 4, 4, 6, 0]
    assert codes[0] == 0x87 and codes[4] == 0x87  # even index low; -0.25 and -0.0 keep the sign
    for e in (-140, -3, 0, 60):
        c, b = oracle.mxfp4_encode(w * 2.0 ** e)
        if e > -127:
            assert np.array_equal(oracle.mxfp4_decode(c, b), oracle.mxfp4_decode(codes, 127) * 2.0 ** e)
        else:
            assert b[0] == 0
    w[5] = np.inf
    c, b = oracle.mxfp4_encode(w)
    assert b[0] == 255 and np.isnan(oracle.mxfp4_decode(c, b)).all()


def test_mxfp4_encode_is_nearest():
    g = np.random.default_rng(1)
    w = g.standard_normal((64, 96)) * 2.0 ** g.integers(-20, 20, (64, 1))
    c, b = oracle.mxfp4_encode(w)
    v = oracle.mxfp4_decode(c, b)
    unit = np.repeat(np.ldexp(1.0, b.astype(int) - 127), 32, axis=1)
    grid = np.concatenate([oracle.mxfp4_oracle.E2M1, -oracle.mxfp4_oracle.E2M1])
    best = np.abs(w[..., None] - grid * unit[..., None]).min(axis=-1)
    assert np.array_equal(np.abs(w - v), best)
    # a second pass gives the codes again where the group kept its largest magnitude's binade
    c2, b2 = oracle.mxfp4_encode(v)
    keep = b2 == b
    assert keep.mean() > 0.9
    assert np.array_equal(oracle.mxfp4_decode(c2, b2)[np.repeat(keep, 32, 1)], v[np.repeat(keep, 32, 1)])


def test_mxfp4_grouped_products_are_the_dense_ones():
    g = np.random.default_rng(2)
    I, H = 32, 64
    c1, s1 = oracle.mxfp4_encode(g.standard_normal((2, 2 * I, H)))
    c2, s2 = oracle.mxfp4_encode(g.standard_normal((2, H, I)))
    x = g.standard_normal((5, H))
    a = oracle.mxfp4_grouped_gate_up(x, [0, 2, 5], c1, s1, I)[0]
    y = oracle.mxfp4_grouped_down(a, [0, 2, 5], c2, s2)[0]
    for r in range(5):
        s = 0 if r < 2 else 1
        w, d = oracle.mxfp4_decode(c1[s], s1[s]), oracle.mxfp4_decode(c2[s], s2[s])
        z = w[:I] @ x[r]
        assert np.allclose(y[r], d @ (z / (1 + np.exp(-z)) * (w[I:] @ x[r])), rtol=1e-12)
