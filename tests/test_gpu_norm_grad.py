"""Layer norm, and the gradients of both norms, on the GPU against the fp64 oracle.

Tolerances, with u = 2^-24. A row's sum passes at most 64 f32 additions (32 in a thread, 2 x 2 more, 6 in the
wave, 16 over the waves). n = (h - mean) r: the deviation carries one rounding, its mean's correction and the
root 64 u of the deviations' mean and of n, so n is within u (64 (|n| + 1) + 4); with a residual h itself is
rounded, 2 u max|h| r more. v = n gamma + beta adds two roundings, y its type's (bf16 2^-8, f32 2^-24).
dx = r (g - mean g - n mean(g n)): each term's rounding, 64 u of the sums' terms, n's error wherever n stands.
dgamma, dbeta: n's error, and at most 176 additions in a chain (79 rows of a block, 16 groups of its waves, 64
blocks and 16 lines of the fold; up to 20000 rows).
"""
import numpy as np
import pytest
import torch

import moe_expert_dispatch_amd as moe
import oracle
from gpu_common import announce, assert_within, device, np64
from oracle import training as tr

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
ROUND = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
TINY = 1e-44
# below its least normal number a type's steps are all one: half of bf16's 2^-133, and of f32's 2^-149 twice (the
# product's and the sum's), which a gradient reaches where the row's deviation is 3e37 (dx some 1e-38)
LEAST = {torch.bfloat16: 2.0 ** -134, torch.float32: 2 * 2.0 ** -150}


def _inputs(T, H, dt, seed):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    x = (n(T, H) + 0.5 * n(T, 1)).to(dt)
    res = (n(T, H) * 3).to(dt)
    gamma, beta = (1 + 0.2 * n(H)).to(dt), (0.3 * n(H)).to(dt)
    return x, res, gamma, beta, (n(T, H) * 0.1).to(dt), (n(T, H) * 0.1).to(dt)


def _n_error(n):
    return U * (64 * (np.abs(n) + 1) + 4)


def _check_forward(y, ro, q, x, gamma, beta, eps, res, scale, what):
    dt = x.dtype
    h, v = tr.layer_norm(x, gamma, beta, eps, res)
    n, r = tr.normalise(h, eps, True)
    gm, bt = np.abs(np64(gamma)), 0.0 if beta is None else np.abs(np64(beta))
    err = _n_error(n)
    if res is not None:
        err = err + 2 * U * np.abs(h).max(1, keepdims=True) * r
        assert_within(np64(ro), h, (ROUND[dt] + 2 * U) * np.abs(h) + TINY, what + " residual")
    err = err * gm + 2 * U * (np.abs(v) + bt)
    assert_within(np64(y), v, err + ROUND[dt] * (np.abs(v) + err) + TINY, what + " y")
    if q is not None:
        inv = np.float64(np.float32(1) / np.float32(scale))
        code = lambda a: oracle.e4m3_decode(oracle.e4m3_encode(np.clip(a * inv, -448, 448)))  # noqa: E731
        got = oracle.e4m3_decode(q.cpu().numpy())
        wide = err + 2 * U * np.abs(v)
        assert ((got >= code(v - wide)) & (got <= code(v + wide))).all(), what + " codes"


def _check_backward(dx, dg, db, dy, x, gamma, eps, centred, dres, what):
    dt = x.dtype
    want, wg, wb = tr.norm_backward(dy, x, gamma, eps, centred, dres)
    n, r = tr.normalise(x, eps, centred)
    d, gm = np64(dy), np64(gamma)
    g, ne = np.abs(d * gm), _n_error(n)
    an = np.abs(n)
    sn = (d * gm * n).mean(1, keepdims=True)
    sn_err = 66 * U * (g * an).mean(1, keepdims=True) + (g * ne).mean(1, keepdims=True)
    err = 3 * U * g + (66 * U * g.mean(1, keepdims=True) if centred else 0) + an * sn_err + ne * np.abs(sn)
    plain = np.abs(r * (g + g.mean(1, keepdims=True) + an * np.abs(sn)))
    err = r * err + 70 * U * plain
    if dres is not None:
        err = err + 2 * U * np.abs(np64(dres))
    if dx is not None:
        assert_within(np64(dx), want, err + ROUND[dt] * (np.abs(want) + err) + LEAST[dt], what + " dx")
    chain = 176 * U
    if dg is not None:
        assert_within(np64(dg), wg, (np.abs(d) * ne).sum(0) + chain * (np.abs(d) * an).sum(0) + TINY, what + " dgamma")
    if db is not None:
        assert_within(np64(db), wb, chain * np.abs(d).sum(0) + TINY, what + " dbeta")


SIZES = [(1, 8), (1, 4096), (3, 504), (5, 520), (2, 8200), (7, 2056), (1, 16392), (2, 32768), (257, 1408),
         (1000, 5120), (33, 64), (100, 128), (41, 136), (70, 256), (19, 264), (2100, 512), (5000, 40)]


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,H", SIZES)
def test_layer_norm(dt, T, H):
    dev = device()
    announce(f"layer_norm {dt} T={T} H={H}")
    x, res, gamma, beta, _, _ = _inputs(T, H, dt, T * 7 + H)
    for rr, bb, scale in ((res, beta, 1 / 56), (None, beta, 0.01), (res, None, None), (None, None, None)):
        y, ro, q = moe.layer_norm(x.to(dev), gamma.to(dev), None if bb is None else bb.to(dev), 1e-5,
                                  None if rr is None else rr.to(dev), scale)
        torch.cuda.synchronize()
        assert (ro is None) == (rr is None) and (q is None) == (scale is None)
        _check_forward(y, ro, q, x, gamma, bb, 1e-5, rr, scale, f"res {rr is not None} scale {scale}")


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,H", SIZES)
def test_backward(dt, T, H):
    dev = device()
    announce(f"norm backward {dt} T={T} H={H}")
    x, _, gamma, _, dy, dres = _inputs(T, H, dt, T * 5 + H)
    X, G, D, R = (t.to(dev) for t in (x, gamma, dy, dres))
    for rr in (None, dres):
        RR = None if rr is None else R
        dx, dg, db = moe.layer_norm_backward(D, X, G, 1e-5, dresidual=RR)
        _check_backward(dx, dg, db, dy, x, gamma, 1e-5, True, rr, f"layer {rr is not None}")
        dx, dg = moe.rms_norm_backward(D, X, G, 1e-5, dresidual=RR)
        _check_backward(dx, dg, None, dy, x, gamma, 1e-5, False, rr, f"rms {rr is not None}")


def test_many_rows():
    """More rows than blocks, the last round not full; runs repeat bit for bit."""
    dev = device()
    for T, H, dt in ((20000, 64, torch.bfloat16), (3333, 1032, torch.float32), (9001, 24, torch.float32)):
        announce(f"norm backward many rows T={T} H={H}")
        x, _, gamma, _, dy, dres = _inputs(T, H, dt, T)
        args = [t.to(dev) for t in (dy, x, gamma)]
        dx, dg, db = moe.layer_norm_backward(*args, 1e-6, dresidual=dres.to(dev))
        _check_backward(dx, dg, db, dy, x, gamma, 1e-6, True, dres, "many")
        again = moe.layer_norm_backward(*args, 1e-6, dresidual=dres.to(dev))
        for u, v in zip(again, (dx, dg, db)):
            assert torch.equal(u, v)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_rows_far_from_zero_and_extreme(dt):
    """A mean far above the deviation; rows whose squares leave f32's range, either way; padded rows of zeros."""
    dev = device()
    announce(f"layer norm extreme rows {dt}")
    for H in (120, 264, 4104):
        g = torch.Generator().manual_seed(H)
        z = torch.randn(8, H, generator=g)
        x = torch.stack([z[0] + 1000, z[1] * 0, z[2] * 1e25, z[3] * 1e-25, z[4] * 1e-4 - 7, z[5] * 1e18 + 1e19,
                         z[6] * 1e-18, 3e37 * torch.sign(z[7])]).to(dt)
        dy, gamma = torch.randn(8, H, generator=g).to(dt), (1 + 0.1 * torch.randn(H, generator=g)).to(dt)
        beta = torch.randn(H, generator=g).to(dt)
        for eps in (1e-5, 1e-30):
            y, _, _ = moe.layer_norm(x.to(dev), gamma.to(dev), beta.to(dev), eps)
            _check_forward(y, None, None, x, gamma, beta, eps, None, None, f"H {H} eps {eps}")
            for centred in (True, False):
                fn = moe.layer_norm_backward if centred else moe.rms_norm_backward
                got = fn(dy.to(dev), x.to(dev), gamma.to(dev), eps)
                _check_backward(got[0], got[1], got[2] if centred else None, dy, x, gamma, eps, centred, None,
                                f"H {H} eps {eps} centred {centred}")


def test_a_nan_stays_in_its_row():
    dev = device()
    x, _, gamma, beta, dy, _ = (t.to(dev) for t in _inputs(6, 136, torch.bfloat16, 3))
    want = moe.layer_norm(x, gamma, beta)[0], moe.layer_norm_backward(dy, x, gamma)[0], moe.rms_norm_backward(dy, x, gamma)[0]
    x[2, 7] = float("nan")
    got = moe.layer_norm(x, gamma, beta)[0], moe.layer_norm_backward(dy, x, gamma)[0], moe.rms_norm_backward(dy, x, gamma)[0]
    keep = torch.tensor([0, 1, 3, 4, 5], device=dev)
    for u, v in zip(got, want):
        assert torch.equal(u[keep], v[keep]) and torch.isnan(u[2]).all()


@pytest.mark.parametrize("H", [64, 1032, 8200])
def test_in_place_and_partial_outputs(H):
    dev = device()
    announce(f"norm backward in place H={H}")
    x, res, gamma, beta, dy, dres = (t.to(dev) for t in _inputs(9, H, torch.bfloat16, 5))
    want = moe.layer_norm(x, gamma, beta, 1e-6, res, 0.02)
    xd, rd = x.clone(), res.clone()
    got = moe.layer_norm(xd, gamma, beta, 1e-6, rd, 0.02, y=xd, residual_out=rd)
    assert got[0] is xd and all(torch.equal(u, v) for u, v in zip(got, want))
    want = moe.layer_norm_backward(dy, x, gamma, 1e-6, dresidual=dres)
    for place in ("dy", "x", "dres"):
        t = {"dy": dy.clone(), "x": x.clone(), "dres": dres.clone()}
        got = moe.layer_norm_backward(t["dy"], t["x"], gamma, 1e-6, dresidual=t["dres"], dx=t[place])
        assert all(torch.equal(u, v) for u, v in zip(got, want)), place
    st = torch.cuda.current_stream().cuda_stream
    ws = torch.empty(moe.norm_backward_workspace_size(9, H), dtype=torch.uint8, device=dev)
    so, P = moe.lib(), lambda t: t.data_ptr()  # noqa: E731
    dx, dg, db = torch.empty_like(x), torch.empty(H, device=dev), torch.empty(H, device=dev)
    args = (P(dy), P(x), P(gamma), P(dres), 1, 9, H, 1e-6)
    assert so.moe_layer_norm_backward(*args, P(dx), None, None, None, 0, st) == 0
    assert so.moe_layer_norm_backward(*args, None, P(dg), None, P(ws), ws.numel(), st) == 0
    assert so.moe_layer_norm_backward(*args, None, None, P(db), P(ws), ws.numel(), st) == 0
    assert torch.equal(dx, want[0]) and torch.equal(dg, want[1]) and torch.equal(db, want[2])


def test_no_rows():
    dev = device()
    x, gamma = torch.empty(0, 64, device=dev), torch.ones(64, device=dev)
    assert moe.layer_norm(x, gamma)[0].shape == (0, 64)
    dg, db = torch.full((64,), 7.0, device=dev), torch.full((64,), 7.0, device=dev)
    dx, dg, db = moe.layer_norm_backward(x, x, gamma, dgamma=dg, dbeta=db)
    assert dx.shape == (0, 64) and not dg.any() and not db.any()
    assert not moe.rms_norm_backward(x, x, gamma)[1].any()


def test_refusals():
    dev = device()
    x, res, gamma, beta, dy, dres = (t.to(dev) for t in _inputs(4, 64, torch.bfloat16, 1))
    for bad in (lambda: moe.layer_norm(x, gamma.float()), lambda: moe.layer_norm(x, gamma, beta.float()),
                lambda: moe.layer_norm(x.half(), gamma.half()),
                lambda: moe.layer_norm_backward(dy.float(), x, gamma),
                lambda: moe.rms_norm_backward(dy, x, gamma, dgamma=torch.empty(64, device=dev).bfloat16())):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: moe.layer_norm(x, gamma[:32]), lambda: moe.layer_norm(x.t(), gamma),
                lambda: moe.layer_norm(x, gamma, residual_out=x), lambda: moe.layer_norm(x, gamma, q=x),
                lambda: moe.layer_norm_backward(dy[:2], x, gamma), lambda: moe.layer_norm_backward(dy, x[0], gamma),
                lambda: moe.rms_norm_backward(dy, x, gamma, dresidual=dres.cpu())):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(RuntimeError):
        moe.layer_norm(x, gamma, eps=-1.0)
    with pytest.raises(RuntimeError):
        moe.rms_norm_backward(dy, x, gamma, eps=float("nan"))
    big = torch.zeros(400, 4096, device=dev)
    with pytest.raises(RuntimeError):
        moe.rms_norm_backward(big, big, big[0], ws=torch.empty(16, dtype=torch.uint8, device=dev))
