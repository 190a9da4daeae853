"""CPU oracle of what stands around the layer (numpy, fp64): the norm of its
input, the router's balance loss, and the router's gradient.

TEST INFRASTRUCTURE, as moe_oracle.py, and from the same pages: [EPMASK]
(the router's softmax and renormalisation), [SLOTS] (per-expert load).
"""
from __future__ import annotations

import numpy as np

from .moe_oracle import _f64, _i64


def rms_norm(x, gamma, eps: float, residual=None):
    """(h, v): h = x + residual, v = h / sqrt(mean(h^2) + eps) * gamma."""
    h = _f64(x) + (0.0 if residual is None else _f64(residual))
    return h, h / np.sqrt((h * h).mean(axis=1, keepdims=True) + eps) * _f64(gamma)


def probabilities(logits) -> np.ndarray:
    """Softmax rows; a row of only -inf is 0."""
    l = _f64(logits)
    m = l.max(axis=1, keepdims=True)
    z = np.exp(l - np.where(np.isneginf(m), 0.0, m))
    s = z.sum(axis=1, keepdims=True)
    return z / np.where(s == 0, 1.0, s)


def _valid(logits, mask) -> np.ndarray:
    return np.ones(logits.shape[0], bool) if mask is None else _i64(mask) != 0


def balance_loss(logits, ids, coef: float, mask=None, counts=None):
    """(loss, counts [E + 1], prob [E]); given counts replace the counted ones."""
    ok = np.nonzero(_valid(logits, mask))[0]
    i = _i64(ids)
    E, K, n = logits.shape[1], i.shape[1], ok.size
    if counts is None:
        counts = np.zeros(E + 1, np.int64)
        for t in ok:
            for e in i[t]:
                if 0 <= e < E:
                    counts[e] += 1
        counts[E] = n
    if n == 0:
        return 0.0, counts, np.zeros(E)
    prob = probabilities(_f64(logits)[ok]).sum(axis=0) / n
    return float(coef * E * (counts[:E] / (n * K) * prob).sum()), counts, prob


def routing_weights(logits, ids, renormalize: bool) -> np.ndarray:
    """w [T, K] of given ids; 0 where an id is outside [0, E)."""
    p, i = probabilities(logits), _i64(ids)
    w = np.zeros(i.shape)
    for t in range(i.shape[0]):
        for k, e in enumerate(i[t]):
            if 0 <= e < p.shape[1]:
                w[t, k] = p[t, e]
        if renormalize and w[t].sum() > 0:
            w[t] /= w[t].sum()
    return w


def route_backward(logits, ids, dw, renormalize: bool, counts=None, coef: float = 0.0,
                   dloss: float = 1.0, mask=None) -> np.ndarray:
    """dlogits by the chain rule through dL/dp and the softmax's Jacobian."""
    l, i = _f64(logits), _i64(ids)
    T, E = l.shape
    K = i.shape[1]
    out = np.zeros((T, E))
    for t in np.nonzero(_valid(logits, mask))[0]:
        p = probabilities(l[t:t + 1])[0]
        dp = np.zeros(E)
        if dw is not None:
            d = _f64(dw)[t]
            sel = [(e, d[k]) for k, e in enumerate(i[t]) if 0 <= e < E]
            total = sum(p[e] for e, _ in sel)
            mean = sum(p[e] * v for e, v in sel)
            for e, v in sel:
                if not renormalize:
                    dp[e] += v
                elif total > 0:
                    dp[e] += v / total - mean / total ** 2
        if counts is not None and counts[E] > 0:
            dp += dloss * coef * E / counts[E] * np.asarray(counts[:E]) / (float(counts[E]) * K)
        out[t] = p * (dp - (p * dp).sum())
    return out
