"""moe_balance_loss and moe_route_backward on the GPU against the fp64 oracle.

Tolerances count f32 roundings, u = 2^-24. A probability: the difference
logit - max rounds once (relative to its size R, the row's range), so the
exponential is off by R u, plus 3 u of its own; the denominator sums positive
terms over at most 16 + 6 additions, the reciprocal and product round once:
EP = (2 R + 2 * 3 + 22 + 4) u with both exponentials. A sum over tokens of
positive terms adds one u for each addition a term passes: 40 over a block's
lane groups, and the block's rounds.
"""
import numpy as np
import pytest
import torch

import moe_expert_dispatch_amd as moe
import oracle
from gpu_common import announce, assert_within, device, np64

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def _case(T, E, K, seed, pad=0.0, skew=1.0, masked_value=float("nan")):
    g = torch.Generator().manual_seed(seed)
    l = torch.randn(T, E, generator=g) * skew + torch.randn(E, generator=g)
    ids = torch.sort(l, dim=1, descending=True, stable=True)[1][:, :K].int()
    dw = torch.randn(T, K, generator=g)
    mask = None
    if pad:
        mask = (torch.rand(T, generator=g) >= pad).to(torch.uint8)
        l[mask == 0] = masked_value
        dw[mask == 0] = masked_value
        ids[mask == 0] = 1 << 30
    return l, ids, dw, mask


def _range(l, mask):
    ok = l if mask is None else l[mask != 0]
    ok = ok[torch.isfinite(ok)]
    return float(ok.max() - ok.min()) if ok.numel() else 0.0


def _dev(dev, *ts):
    return [None if t is None else t.to(dev) for t in ts]


def _check_loss(dev, l, ids, mask, coef, what):
    T, E = l.shape
    loss, counts, prob = moe.balance_loss(*_dev(dev, l, ids), coef, token_mask=_dev(dev, mask)[0])
    torch.cuda.synchronize()
    w_loss, w_counts, w_prob = oracle.balance_loss(l, ids, coef, mask)
    assert np.array_equal(counts.cpu().numpy(), w_counts), what
    rounds = -(-T // 256)
    rel = (2 * _range(l, mask) + 32 + 40 + rounds) * U
    assert (np.abs(np64(prob) - w_prob) <= rel * w_prob + 1e-38).all(), what
    assert abs(float(loss) - w_loss) <= (rel + 4 * U) * abs(w_loss) + 1e-38, what
    return counts


def _check_grad(dev, l, ids, dw, mask, renorm, counts, coef, dloss, what):
    """|error| <= eps * (the sum of the magnitudes that make up an element): every factor is
    within EP, each of the two dot products adds K or E additions, and the terms a handful more."""
    T, E = l.shape
    K = ids.shape[1]
    got = moe.route_backward(*_dev(dev, l, ids, dw), renorm, counts=counts, coef=coef,
                             dloss=None if dloss is None else torch.tensor(dloss, device=dev),
                             token_mask=_dev(dev, mask)[0])
    torch.cuda.synchronize()
    c = None if counts is None else counts.cpu().numpy().astype(np.int64)
    args = (renorm, c, coef, 1.0 if dloss is None else dloss, mask)
    want = oracle.route_backward(l, ids, dw, *args)
    ok = np.ones(T, bool) if mask is None else mask.numpy() != 0
    p = np.zeros((T, E))
    p[ok] = oracle.layer_oracle.probabilities(l[torch.from_numpy(ok)])
    size = np.zeros((T, E))
    if dw is not None:
        safe = l.clone()
        safe[~torch.from_numpy(ok)] = 0.0
        w = oracle.routing_weights(safe, ids, renorm)
        a = w * np.abs(np64(dw))
        dot = np.nansum(a, axis=1, keepdims=True)
        # renormalised, an expert outside the K has exactly no gradient, and the oracle's sum over
        # the Jacobian leaves the rounding of 64 bits there: 2 E additions of 2^-53, over eps below
        size += (2 * E * 2.0 ** -53 / (34 * U)) * p * 2 * dot
        for t in np.nonzero(ok)[0]:
            if renorm:
                for k in range(K):
                    if 0 <= ids[t, k] < E:
                        size[t, int(ids[t, k])] += a[t, k] + w[t, k] * dot[t, 0]
            else:
                size[t] += p[t] * dot[t, 0]
                for k in range(K):
                    if 0 <= ids[t, k] < E:
                        size[t, int(ids[t, k])] += a[t, k]
    if c is not None and c[E] > 0:
        f = c[:E] / (c[E] * K)
        size += abs(args[2] * args[3]) * E / c[E] * p * (f + (p * f).sum(1, keepdims=True))
    eps = (2 * (2 * _range(l, mask) + 32) + K + 22 + 12) * U
    g = np64(got)
    assert not g[~ok].any(), what
    bad = np.abs(g - want) > eps * size + 1e-38
    assert not bad.any(), (what, int(bad.sum()), np.abs(g - want)[bad].max())
    return got


CASES = [(1, 1, 1), (1, 8, 2), (64, 8, 2), (1000, 7, 7), (333, 60, 4), (129, 64, 9), (77, 128, 16),
         (50, 160, 6), (31, 256, 8), (2, 256, 32), (40, 300, 32), (19, 513, 3), (9, 1024, 8),
         (9000, 60, 4)]


@pytest.mark.parametrize("T,E,K", CASES)
@pytest.mark.parametrize("pad", [0.0, 0.3])
def test_against_oracle(T, E, K, pad):
    dev = device()
    announce(f"router grad T={T} E={E} K={K} pad={pad}")
    l, ids, dw, mask = _case(T, E, K, T + E + K, pad)
    counts = _check_loss(dev, l, ids, mask, 0.02, "loss")
    for renorm in (False, True):
        _check_grad(dev, l, ids, dw, mask, renorm, counts, 0.02, None, f"both renorm={renorm}")
        _check_grad(dev, l, ids, dw, mask, renorm, None, 0.0, None, f"weights renorm={renorm}")
    _check_grad(dev, l, ids, None, mask, False, counts, 0.02, -2.5, "loss only")


def test_gradient_is_a_difference():
    """The derivative of (w * dw).sum() + loss along a random direction, by central differences of
    the oracle's value in 64 bits: step 1e-4, truncation under 1e-8 of second-order-one terms."""
    dev = device()
    announce("router grad differences")
    l, ids, dw, mask = _case(20, 12, 3, 5, 0.2, masked_value=0.0)
    ids[mask == 0] = 0
    coef = 0.5
    _, counts, _ = moe.balance_loss(*_dev(dev, l, ids), coef, token_mask=mask.to(dev))
    c = counts.cpu().numpy().astype(np.int64)
    ok = mask.numpy() != 0
    for renorm in (False, True):
        g = np64(moe.route_backward(*_dev(dev, l, ids, dw), renorm, counts=counts, coef=coef,
                                    token_mask=mask.to(dev)))
        rng = np.random.default_rng(1)
        for _ in range(5):
            d = rng.standard_normal(l.shape)

            def value(h):
                x = np64(l) + h * d
                w = oracle.routing_weights(x, ids, renorm)[ok]
                return (w * np64(dw)[ok]).sum() + oracle.balance_loss(x, ids, coef, mask, c)[0]
            slope = (value(1e-4) - value(-1e-4)) / 2e-4
            assert abs(slope - (g * d).sum()) <= 1e-6 + 200 * U * np.abs(g * d).sum()


@pytest.mark.parametrize("low", [float("-inf"), torch.finfo(torch.float32).min])
def test_rows_with_forbidden_experts(low):
    dev = device()
    announce(f"router grad forbidden experts {low}")
    T, E, K = 40, 24, 3
    l, ids, dw, _ = _case(T, E, K, 11)
    l[:, ::2] = low                       # half of the experts forbidden
    l[7] = low                            # a row that leaves nothing
    ids = torch.sort(l, dim=1, descending=True, stable=True)[1][:, :K].int()
    if low == float("-inf"):
        counts = _check_loss(dev, l, ids, None, 1.0, "loss")
        for renorm in (False, True):
            got = _check_grad(dev, l, ids, dw, None, renorm, counts, 1.0, None, "grad")
            assert not got[7].any()
    else:
        # the range of the finite logits is that of the type: compare with -inf in its place, but
        # the row of equal lowest values is an even one
        counts = moe.balance_loss(*_dev(dev, l, ids), 1.0)[1]
        rest = [t for t in range(T) if t != 7]
        inf = l.clone()
        inf[:, ::2] = float("-inf")
        for renorm in (False, True):
            a = moe.route_backward(*_dev(dev, l, ids, dw), renorm, counts=counts, coef=1.0)
            b = moe.route_backward(*_dev(dev, inf, ids, dw), renorm, counts=counts, coef=1.0)
            assert torch.equal(a[rest], b[rest])
            assert torch.isfinite(a).all()


def test_foreign_and_repeated_ids():
    dev = device()
    announce("router grad foreign ids")
    l, ids, dw, _ = _case(30, 10, 4, 3)
    ids[0] = -1
    ids[1] = 10
    ids[2] = torch.tensor([3, 3, 3, -5], dtype=torch.int32)
    ids[3] = torch.tensor([1, 2, 1, 2 ** 31 - 1], dtype=torch.int32)
    dw[0] = float("inf")                  # pairs that select nothing have no influence
    counts = _check_loss(dev, l, ids, None, 1.0, "loss")
    dw[0] = 7.0
    for renorm in (False, True):
        _check_grad(dev, l, ids, dw, None, renorm, counts, 1.0, None, f"renorm={renorm}")
    dw[0] = float("inf")
    assert torch.isfinite(moe.route_backward(*_dev(dev, l, ids, dw), True)).all()


def test_nothing_valid_and_empty():
    dev = device()
    announce("router grad nothing valid")
    l, ids, dw, mask = _case(50, 16, 2, 3, 0.5)
    mask[:] = 0
    loss, counts, prob = moe.balance_loss(*_dev(dev, l, ids), 1.0, token_mask=mask.to(dev))
    assert float(loss) == 0.0 and not counts.any() and not prob.any()
    assert not moe.route_backward(*_dev(dev, l, ids, dw), True, counts=counts, coef=1.0,
                                  token_mask=mask.to(dev)).any()
    loss, counts, prob = moe.balance_loss(l[:0].to(dev), ids[:0].to(dev), 1.0)
    assert float(loss) == 0.0 and not counts.any() and not prob.any()
    assert moe.route_backward(l[:0].to(dev), ids[:0].to(dev), dw[:0].to(dev), True).shape == (0, 16)


def test_counts_are_exact_and_runs_repeat():
    """A big batch: integer counts exact, loss and probabilities the same bits every time, on
    another stream too, with a workspace of the caller."""
    dev = device()
    announce("balance loss repeat")
    g = torch.Generator(device=dev).manual_seed(2)
    T, E, K = 70001, 96, 5
    l = torch.randn(T, E, generator=g, device=dev)
    ids = torch.randint(0, E, (T, K), generator=g, device=dev, dtype=torch.int32)
    first = moe.balance_loss(l, ids, 1.0)
    assert torch.equal(first[1][:E], torch.bincount(ids.flatten(), minlength=E).int())
    assert int(first[1][E]) == T
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        ws = torch.empty(moe.balance_loss_workspace_size(T, E, K), dtype=torch.uint8, device=dev)
        again = moe.balance_loss(l, ids, 1.0, ws=ws)
    torch.cuda.current_stream().wait_stream(s)
    for a, b in zip(first, again):
        assert torch.equal(a, b)


def test_router_step_captured_in_a_graph():
    """route -> balance_loss -> route_backward as a training step runs them, captured and replayed on
    new inputs with eager work between: every replay gives the eager result."""
    dev = device()
    announce("router step graph")
    T, E, K = 500, 60, 4
    l, _, dw, mask = _case(T, E, K, 1, 0.25, masked_value=0.0)
    l, dw, mask = _dev(dev, l, dw, mask)
    ids = torch.empty(T, K, dtype=torch.int32, device=dev)
    w = torch.empty(T, K, device=dev)

    def step():
        moe.route(l, K, True, ids=ids, w=w)
        loss, counts, prob = moe.balance_loss(l, ids, 0.1, token_mask=mask)
        return loss, counts, prob, moe.route_backward(l, ids, dw, True, counts=counts, coef=0.1,
                                                      token_mask=mask)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(4):
        g = torch.Generator(device=dev).manual_seed(i)
        l.copy_(torch.randn(T, E, generator=g, device=dev))
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in out]
        for a, b in zip(got, step()):
            assert torch.equal(a, b)


def test_refusals():
    dev = device()
    l, ids, dw, _ = _case(6, 8, 2, 1)
    l, ids, dw = _dev(dev, l, ids, dw)
    for bad in (lambda: moe.balance_loss(l.double(), ids, 1.0),
                lambda: moe.balance_loss(l, ids.long(), 1.0),
                lambda: moe.route_backward(l, ids, dw.double(), True)):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: moe.balance_loss(l, ids[:3], 1.0),
                lambda: moe.balance_loss(l[0], ids, 1.0),
                lambda: moe.balance_loss(l, ids, 1.0, token_mask=torch.ones(5, dtype=torch.uint8, device=dev)),
                lambda: moe.route_backward(l, ids, dw[:, :1].contiguous(), True),
                lambda: moe.route_backward(l, ids, dw, True, counts=torch.zeros(8, dtype=torch.int32, device=dev)),
                lambda: moe.route_backward(l, ids, dw, True, dloss=torch.zeros(2, device=dev)),
                lambda: moe.route_backward(l.t(), ids, dw, True)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(RuntimeError):
        moe.route_backward(l, ids, None, True)
    with pytest.raises(RuntimeError):
        moe.balance_loss(l, ids, 1.0, ws=torch.empty(8, dtype=torch.uint8, device=dev))


# ------------------------------------------------------------------ every element a number
def _grad_within(dev, l, ids, dw, mask, renorm, counts, coef, what):
    """As _check_grad, in a form that no NaN passes, for finite or -inf logits and finite dw."""
    T, E = l.shape
    K = ids.shape[1]
    got = np64(moe.route_backward(*_dev(dev, l, ids, dw), renorm, counts=counts, coef=coef,
                                  token_mask=_dev(dev, mask)[0]))
    c = None if counts is None else counts.cpu().numpy().astype(np.int64)
    ok = np.ones(T, bool) if mask is None else mask.numpy() != 0
    keep = torch.from_numpy(ok)
    want, size = np.zeros((T, E)), np.zeros((T, E))
    l, ids, dw = l[keep], ids[keep], None if dw is None else dw[keep]
    want[ok] = oracle.route_backward(l, ids, dw, renorm, c, coef, 1.0)
    p = oracle.layer_oracle.probabilities(l)
    s = np.zeros_like(p)
    if dw is not None:
        w = oracle.routing_weights(l, ids, renorm)
        a = w * np.abs(np64(dw))
        dot = a.sum(1, keepdims=True)
        # what the 64 bits of the reference leave where its terms cancel (see _check_grad)
        s += (2 * E * 2.0 ** -53 / (34 * U)) * p * 2 * dot
        if not renorm:
            s += p * dot
        i = ids.numpy()
        for t, k in zip(*np.nonzero((i >= 0) & (i < E))):
            s[t, i[t, k]] += a[t, k] + (w[t, k] * dot[t, 0] if renorm else 0.0)
    if c is not None and c[E] > 0:
        f = c[:E] / (c[E] * K)
        s += abs(coef) * E / c[E] * p * (f + (p * f).sum(1, keepdims=True))
    size[ok] = s
    eps = (2 * (2 * _range(l, None) + 32) + K + 22 + 12) * U
    assert_within(got, want, eps * size + ok[:, None] * 1e-38, what)


@pytest.mark.parametrize("T,E,K", CASES)
@pytest.mark.parametrize("pad", [0.0, 0.3])
def test_gradient_is_a_number_everywhere(T, E, K, pad):
    dev = device()
    announce(f"router grad numbers T={T} E={E} K={K} pad={pad}")
    l, ids, dw, mask = _case(T, E, K, 7 * T + E + K, pad)
    counts = moe.balance_loss(*_dev(dev, l, ids), 0.02, token_mask=_dev(dev, mask)[0])[1]
    for renorm in (False, True):
        _grad_within(dev, l, ids, dw, mask, renorm, counts, 0.02, f"both renorm={renorm}")
        _grad_within(dev, l, ids, dw, mask, renorm, None, 0.0, f"weights renorm={renorm}")
    _grad_within(dev, l, ids, None, mask, False, counts, 0.02, "loss only")


@pytest.mark.parametrize("E,K", [(8, 2), (60, 4), (256, 8), (1000, 8)])
def test_gradient_is_a_number_beside_forbidden_and_foreign(E, K):
    """Experts at -inf, whole rows of them, selected ones among them, foreign and repeated ids."""
    dev = device()
    announce(f"router grad numbers forbidden E={E} K={K}")
    T = 64
    l, ids, dw, _ = _case(T, E, K, E)
    l[:, ::2] = float("-inf")
    l[5] = float("-inf")
    l[6, 1:] = float("-inf")
    l[6, 0] = 0.25
    ids = torch.sort(l, dim=1, descending=True, stable=True)[1][:, :K].int()
    ids[8] = 0                                   # a forbidden expert alone, K times
    ids[9, 0] = 2                                # and one beside others
    ids[10] = -1
    ids[11, -1] = E
    ids[12] = ids[12, 0]
    for coef, loss in ((1.0, True), (0.0, False)):
        counts = moe.balance_loss(*_dev(dev, l, ids), 1.0)[1] if loss else None
        for renorm in (False, True):
            _grad_within(dev, l, ids, dw, None, renorm, counts, coef, f"loss={loss} renorm={renorm}")


def test_gradient_repeats_with_an_expert_held_many_times():
    """Terms of one expert held up to 32 times are added in LDS: the same bits every time."""
    dev = device()
    announce("router grad repeated ids")
    g = torch.Generator(device=dev).manual_seed(9)
    for E, K in ((8, 8), (64, 16), (256, 32), (700, 32)):
        l = torch.randn(500, E, generator=g, device=dev)
        dw = torch.randn(500, K, generator=g, device=dev)
        ids = torch.randint(0, 3, (500, K), generator=g, device=dev, dtype=torch.int32)
        first = moe.route_backward(l, ids, dw, False)
        for _ in range(20):
            assert torch.equal(moe.route_backward(l, ids, dw, False), first)


def test_most_tokens():
    """2^31 - 1 tokens of one expert, the most that T * K < 2^31 allows: the loss, its counts and an exactly
    zero gradient (a softmax of one is constant)."""
    dev = device()
    announce("router 2^31 - 1 tokens")
    if torch.cuda.mem_get_info()[0] < 45 * 2 ** 30:
        pytest.skip("needs 45 GiB of device memory")
    T = 2 ** 31 - 1
    l = torch.full((T, 1), 0.5, device=dev)
    ids = torch.zeros(T, 1, dtype=torch.int32, device=dev)
    d = torch.full((T, 1), 7.0, device=dev)
    loss, counts, prob = moe.balance_loss(l, ids, 0.25)
    assert counts.tolist() == [T, T] and float(prob) == 1.0 and float(loss) == 0.25
    for renorm in (False, True):
        d.fill_(7.0)
        moe.route_backward(l, ids, l, renorm, counts=counts, coef=0.25, dlogits=d)
        assert float(d.abs().max()) == 0.0
    del l, ids, d
    torch.cuda.empty_cache()
