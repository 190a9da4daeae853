"""fp64 formulas of the layer's training pass: norms and their gradients, the gradients of the
weighted sum and of the permutation, of the SwiGLU and of the experts' products. numpy only."""
import numpy as np


def _f64(a):
    return None if a is None else np.asarray(getattr(a, "detach", lambda: a)().cpu().double().numpy()
                                             if hasattr(a, "cpu") else a, dtype=np.float64)


def normalise(x, eps, centred):
    """(n, r): each row's deviation over its standard deviation, and 1 / that."""
    x = _f64(x)
    c = x - x.mean(1, keepdims=True) if centred else x
    r = 1.0 / np.sqrt((c * c).mean(1, keepdims=True) + eps)
    return c * r, r


def layer_norm(x, gamma, beta, eps, residual=None):
    """(h, v) before their rounding."""
    h = _f64(x) + (0.0 if residual is None else _f64(residual))
    n, _ = normalise(h, eps, True)
    return h, n * _f64(gamma) + (0.0 if beta is None else _f64(beta))


def norm_backward(dy, x, gamma, eps, centred, dresidual=None):
    """(dx, dgamma, dbeta) before their rounding."""
    dy, gamma = _f64(dy), _f64(gamma)
    n, r = normalise(x, eps, centred)
    g = dy * gamma
    dx = g - n * (g * n).mean(1, keepdims=True)
    if centred:
        dx = dx - g.mean(1, keepdims=True)
    dx = r * dx + (0.0 if dresidual is None else _f64(dresidual))
    return dx, (dy * n).sum(0), dy.sum(0)


def combine_backward(dout, y, pair_row, w, K):
    """(dy of the rows that some pair has, else 0; dw [T, K]); w None: weight 1."""
    dout, y, pr = _f64(dout), _f64(y), np.asarray(pair_row).reshape(-1)
    w = np.ones(pr.size) if w is None else _f64(w).reshape(-1)
    dy, dw = np.zeros_like(y), np.zeros(pr.size)
    for p, row in enumerate(pr):
        if row >= 0:
            dy[row] = w[p] * dout[p // K]
            dw[p] = dout[p // K] @ y[row]
    return dy, dw.reshape(-1, K)


def permute_backward(dx_perm, pair_row, K, w=None, x=None):
    """(dx [T, H], dw [T, K] or None)."""
    d, pr = _f64(dx_perm), np.asarray(pair_row).reshape(-1)
    T = pr.size // K
    wt = np.ones(pr.size) if w is None else _f64(w).reshape(-1)
    dx, dw = np.zeros((T, d.shape[1])), np.zeros(pr.size)
    for p, row in enumerate(pr):
        if row >= 0:
            dx[p // K] += wt[p] * d[row]
            if x is not None:
                dw[p] = d[row] @ _f64(x[p // K])
    return dx, None if x is None else dw.reshape(-1, K)


def sigmoid(g):
    return np.where(g >= 0, 1.0 / (1.0 + np.exp(-np.abs(g))), np.exp(-np.abs(g)) / (1.0 + np.exp(-np.abs(g))))


def swiglu(h):
    h = _f64(h)
    I = h.shape[1] // 2
    return h[:, :I] * sigmoid(h[:, :I]) * h[:, I:]


def swiglu_backward(h, dact):
    h, d = _f64(h), _f64(dact)
    I = h.shape[1] // 2
    g, u = h[:, :I], h[:, I:]
    s = sigmoid(g)
    return np.concatenate([d * u * s * (1.0 + g * (1.0 - s)), d * g * s], 1)


def grouped_rows_grad(dc, offsets, w):
    """dc[r] w[s] for the rows of each slot; 0 behind the last."""
    dc, w = _f64(dc), _f64(w)
    out = np.zeros((dc.shape[0], w.shape[2]))
    for s in range(w.shape[0]):
        out[offsets[s]:offsets[s + 1]] = dc[offsets[s]:offsets[s + 1]] @ w[s]
    return out


def grouped_weight_grad(dc, a, offsets):
    dc, a = _f64(dc), _f64(a)
    S = len(offsets) - 1
    return np.stack([dc[offsets[s]:offsets[s + 1]].T @ a[offsets[s]:offsets[s + 1]] for s in range(S)])
