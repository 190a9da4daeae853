"""CPU oracle of the MXFP4 expert path (numpy, fp64).

TEST INFRASTRUCTURE, as moe_oracle.py. Page: [A2A] review of torch_moe.py
(quantized MoE ops run the same routed template with 4-bit expert linears);
the format is the OCP microscaling specification's MXFP4: E2M1 elements in
groups of 32 under one E8M0 scale. Readings: the scale of a group is
2^(floor(log2 amax) - 2), not below 2^-127; elements round to nearest, ties
to the even code, and saturate at 6; a group with a non-finite value is NaN;
two codes a byte, the even index in the low four bits.
"""
from __future__ import annotations

import numpy as np

from .moe_oracle import _f64, silu

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def _u8(a) -> np.ndarray:
    return a.detach().cpu().numpy() if hasattr(a, "detach") else np.asarray(a, dtype=np.uint8)


def mxfp4_decode(codes, scale) -> np.ndarray:
    """Values [..., K] of codes [..., K/2] and scales [..., K/32]."""
    c, b = _u8(codes), _u8(scale).astype(np.int64)
    nib = np.stack([c & 15, c >> 4], axis=-1).reshape(*c.shape[:-1], -1)
    v = np.where(nib >= 8, -1.0, 1.0) * E2M1[nib & 7]
    s = np.where(b == 255, np.nan, np.ldexp(1.0, b - 127))
    return (v.reshape(*b.shape, 32) * s[..., None]).reshape(nib.shape)


def mxfp4_encode(w):
    """(codes [..., K/2], scales [..., K/32]) of w [..., K]: the nearest element
    among the eight magnitudes by a search over their midpoints."""
    w = _f64(w)
    g = w.reshape(*w.shape[:-1], -1, 32)
    amax = np.abs(g).max(axis=-1)
    bad = ~np.isfinite(amax)
    _, e = np.frexp(np.where(bad | (amax == 0), 1.0, amax))  # amax in [2^(e-1), 2^e)
    b = np.where(amax == 0, 0, np.maximum(e - 1 - 2 + 127, 0))
    a = np.abs(np.where(bad[..., None], 0.0, g)) / np.ldexp(1.0, b - 127)[..., None]
    mid = (E2M1[1:] + E2M1[:-1]) / 2
    lo = np.searchsorted(mid, a, side="left")    # a midpoint goes down
    hi = np.searchsorted(mid, a, side="right")   # a midpoint goes up
    code = np.where(lo % 2 == 0, lo, hi)         # of the two the even one
    code = code + 8 * np.signbit(g)
    b = np.where(bad, 255, b).astype(np.uint8)
    code = code.reshape(w.shape).astype(np.uint8)
    return code[..., 0::2] | (code[..., 1::2] << 4), b


def mxfp4_grouped_gate_up(a, offsets, codes, scale, I: int):
    """([rows, I] of silu(a Wg^T) * (a Wu^T), and g, u and the sums of the
    products' magnitudes behind them) for the rows of every slot."""
    a = _f64(a)
    off = np.asarray(offsets, dtype=np.int64)
    g, u = np.zeros((a.shape[0], I)), np.zeros((a.shape[0], I))
    gm, um = np.zeros_like(g), np.zeros_like(u)
    for s in range(off.size - 1):
        r = slice(off[s], off[s + 1])
        if off[s + 1] > off[s]:
            w = mxfp4_decode(codes[s], scale[s])
            g[r], u[r] = a[r] @ w[:I].T, a[r] @ w[I:].T
            gm[r], um[r] = np.abs(a[r]) @ np.abs(w[:I]).T, np.abs(a[r]) @ np.abs(w[I:]).T
    return silu(g) * u, g, u, gm, um


def mxfp4_grouped_down(a, offsets, codes, scale):
    """([rows, H] of a Wd^T, and the sums of the products' magnitudes)."""
    a = _f64(a)
    off = np.asarray(offsets, dtype=np.int64)
    y = np.zeros((a.shape[0], codes.shape[1]))
    m = np.zeros_like(y)
    for s in range(off.size - 1):
        r = slice(off[s], off[s + 1])
        if off[s + 1] > off[s]:
            w = mxfp4_decode(codes[s], scale[s])
            y[r], m[r] = a[r] @ w.T, np.abs(a[r]) @ np.abs(w).T
    return y, m
