"""moe_rms_norm on the GPU against the fp64 oracle.

Tolerance: h carries one f32 rounding; the sum of squares has only positive
terms, each passing at most 36 f32 additions in a thread (4 vectors of 8 and
4 more), 6 in the wave and 16 over the waves, so its relative error is under
64 * 2^-24, its root's half of that; root, quotient and two products round
once each. So v is within 64 * 2^-24 of the oracle's, relative. y adds its
type's rounding (bf16 2^-8, f32 2^-24). A code has to be the rounding of
some value within that bound of v / scale.
"""
import numpy as np
import pytest
import torch

import moe_expert_dispatch_amd as moe
import oracle
from gpu_common import announce, assert_close, device, np64

pytestmark = pytest.mark.gpu

V_REL = 64 * 2.0 ** -24
ROUND = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def _inputs(T, H, dt, seed, residual=True):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, H, generator=g).to(dt)
    r = (torch.randn(T, H, generator=g) * 3).to(dt) if residual else None
    gamma = (1 + 0.2 * torch.randn(H, generator=g)).to(dt)
    return x, r, gamma


def _check(y, ro, q, x, r, gamma, eps, scale, what):
    dt = x.dtype
    h, v = oracle.rms_norm(x, gamma, eps, r)
    if ro is not None:
        assert_close(np64(ro), h, (ROUND[dt] + 2 * 2.0 ** -24, 1e-44), what + " residual")
    assert_close(np64(y), v, (ROUND[dt] + 2 * V_REL, 1e-40), what + " y")
    if q is not None:
        inv = np.float64(np.float32(1) / np.float32(scale))
        a, b = v * inv * (1 - 2 * V_REL), v * inv * (1 + 2 * V_REL)
        lo = oracle.e4m3_decode(oracle.e4m3_encode(np.clip(np.minimum(a, b), -448, 448)))
        hi = oracle.e4m3_decode(oracle.e4m3_encode(np.clip(np.maximum(a, b), -448, 448)))
        got = oracle.e4m3_decode(q.cpu().numpy())
        assert ((got >= lo) & (got <= hi)).all(), what + " codes"


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,H", [(1, 8), (1, 4096), (3, 504), (5, 520), (2, 8200), (7, 2056),
                                 (1, 16392), (2, 32768), (257, 1408), (1000, 5120), (33, 64)])
def test_norm_against_oracle(dt, T, H):
    dev = device()
    announce(f"rms_norm {dt} T={T} H={H}")
    x, r, gamma = _inputs(T, H, dt, T * 7 + H)
    for res, scale in ((r, 1 / 56), (None, 0.01), (r, None), (None, None)):
        y, ro, q = moe.rms_norm(x.to(dev), gamma.to(dev), 1e-5, None if res is None else res.to(dev),
                                scale)
        torch.cuda.synchronize()
        assert (ro is None) == (res is None) and (q is None) == (scale is None)
        _check(y, ro, q, x, res, gamma, 1e-5, scale, f"res {res is not None} scale {scale}")


def test_norm_in_place_and_partial_outputs():
    dev = device()
    announce("rms_norm in place")
    x, r, gamma = _inputs(9, 1032, torch.bfloat16, 5)
    want = moe.rms_norm(x.to(dev), gamma.to(dev), 1e-6, r.to(dev), 0.02)
    xd, rd = x.to(dev), r.to(dev)
    y, ro, q = moe.rms_norm(xd, gamma.to(dev), 1e-6, rd, 0.02, y=xd, residual_out=rd)
    assert y is xd and ro is rd
    for a, b in zip((y, ro, q), want):
        assert torch.equal(a, b)
    # only the codes, only the sum: the C ABI's optional outputs
    q2 = torch.empty_like(q)
    st = torch.cuda.current_stream().cuda_stream
    a, b, c = x.to(dev), r.to(dev), gamma.to(dev)
    assert moe.lib().moe_rms_norm(a.data_ptr(), b.data_ptr(), c.data_ptr(), 1, 9, 1032, 1e-6, None,
                                  None, q2.data_ptr(), 0.02, st) == 0
    s2 = torch.empty_like(a)
    assert moe.lib().moe_rms_norm(a.data_ptr(), b.data_ptr(), c.data_ptr(), 1, 9, 1032, 1e-6,
                                  s2.data_ptr(), None, None, 0.0, st) == 0
    assert torch.equal(q2, want[2]) and torch.equal(s2, want[1])


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_norm_extreme_rows(dt):
    dev = device()
    announce(f"rms_norm extreme rows {dt}")
    H = 264
    x = torch.ones(5, H)
    x[0] = 0.0                 # a padded row: all zero, eps keeps it zero
    x[1] = 1e-20               # far below eps
    x[2] = 1e17                # squares near the top of f32: 1e34 * 264 < 3.4e38
    x[3, 5] = 1e15             # one channel carries the norm
    x[4, 7] = float("nan")     # stays in its row
    x, gamma = x.to(dt), torch.full((H,), 2.0).to(dt)
    y, _, q = moe.rms_norm(x.to(dev), gamma.to(dev), 1e-6, q_scale=1.0)
    y = y.cpu()
    assert not y[0].any() and not q[0].cpu().any()
    _check(y[1:4], None, None, x[1:4], None, gamma, 1e-6, None, "extreme")
    assert torch.isnan(y[4]).all()


def test_norm_refusals():
    dev = device()
    x, r, gamma = (t.to(dev) for t in _inputs(4, 64, torch.bfloat16, 1))
    for bad in (lambda: moe.rms_norm(x, gamma.float()),
                lambda: moe.rms_norm(x, gamma, residual=r.float()),
                lambda: moe.rms_norm(x.half(), gamma.half())):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: moe.rms_norm(x, gamma[:32].contiguous()),
                lambda: moe.rms_norm(x.t(), gamma),
                lambda: moe.rms_norm(x, gamma, residual=r[:2]),
                lambda: moe.rms_norm(x, gamma, residual_out=r),
                lambda: moe.rms_norm(x, gamma, q=torch.empty(4, 64, dtype=torch.uint8, device=dev)),
                lambda: moe.rms_norm(x[0], gamma)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(RuntimeError):
        moe.rms_norm(x[:, :60].contiguous(), gamma[:60].contiguous())
    with pytest.raises(RuntimeError):
        moe.rms_norm(x, gamma, q_scale=float("nan"))
    y, _, _ = moe.rms_norm(x[:0], gamma)
    assert y.shape == (0, 64)


def test_norm_feeds_the_fp8_layer():
    """forward with x_codes takes q as it is: bit for bit the result of the
    bf16 input whose quantisation gives the same codes."""
    dev = device()
    announce("rms_norm -> forward fp8 x_codes")
    T, H, I, E, K, a1 = 37, 256, 256, 6, 2, 1 / 32
    g = torch.Generator().manual_seed(8)
    x, r, gamma = _inputs(T, H, torch.bfloat16, 9)
    y, _, q = moe.rms_norm(x.to(dev), gamma.to(dev), 1e-6, r.to(dev), a1)
    codes = lambda *s: (torch.randint(0x20, 0x40, s, generator=g, dtype=torch.uint8) |  # noqa: E731
                        (torch.randint(0, 2, s, generator=g, dtype=torch.uint8) << 7)).to(dev)
    wgu, wd = codes(E, 2 * I, H), codes(E, H, I)
    sc = torch.full((E,), 1 / 16, device=dev)
    logits = torch.randn(T, E, generator=g).to(dev)
    shared = torch.randn(T, H, generator=g).bfloat16().to(dev)
    cfg = dict(T=T, H=H, I=I, E_global=E, K=K, renormalize=True, S=E, dtype=moe.FP8, a1_scale=a1,
               a2_scale=0.25)
    kw = dict(logits=logits, w_gate_up_scale=sc, w_down_scale=sc, shared_out=shared)
    got = moe.forward(moe.ForwardConfig(**cfg, x_codes=True), q, wgu, wd, **kw)
    # the values the codes stand for are bf16 numbers, and quantise to the same codes
    xb = (q.view(torch.float8_e4m3fn).float() * a1).bfloat16()
    assert torch.equal(moe.quantize_fp8(xb, a1), q)
    want = moe.forward(moe.ForwardConfig(**cfg), xb, wgu, wd, **kw)
    assert torch.equal(got, want) and got.abs().sum() > 0
    with pytest.raises(TypeError):
        moe.forward(moe.ForwardConfig(**cfg, x_codes=True), y, wgu, wd, **kw)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("eps", [0.0, 1e-42, 1e-30])
def test_norm_of_rows_whose_squares_leave_f32(dt, eps):
    """Rows whose squares are below or above f32's range, against the formula; the tolerance is that of every
    other row, since the sum is kept in 64 bits there (and h * h is exact in them)."""
    dev = device()
    announce(f"rms_norm squares out of range {dt} eps={eps}")
    g = torch.Generator().manual_seed(3)
    for H in (8, 264, 8200, 32768):
        sizes = torch.tensor([1e-19, 1e-21, 1e-23, 1e-25, 1e-30, 1e-37, 1e-39, 1e19, 1e25, 1e37, 1.0])
        x = torch.randn(len(sizes), H, generator=g).clamp(-8, 8) * sizes[:, None]
        x[3, 5] = 1e-12                 # one channel carries the norm
        x[8, 2:] = 1e-25                # squares that overflow beside squares that underflow
        r = (0.5 * x).to(dt)
        x, gamma = x.to(dt), (1 + 0.2 * torch.randn(H, generator=g)).to(dt)
        for res in (None, r):
            y, ro, q = moe.rms_norm(x.to(dev), gamma.to(dev), eps, None if res is None else res.to(dev), 1 / 56)
            _check(y, ro, q, x, res, gamma, float(np.float32(eps)), 1 / 56, f"H={H} res={res is not None}")


def test_norm_of_more_rows_than_a_grid_line_has_threads_for():
    """2^26 + 3 rows: with 64 threads a row past the 2^32 threads of one grid dimension."""
    dev = device()
    announce("rms_norm 2^26 + 3 rows")
    T, H = 2 ** 26 + 3, 8
    x = torch.arange(T * H, device=dev, dtype=torch.int32).remainder_(251).sub_(125).to(torch.bfloat16).view(T, H)
    gamma = torch.ones(H, dtype=torch.bfloat16, device=dev)
    y, _, q = moe.rms_norm(x, gamma, 1e-6, q_scale=1 / 56)
    # the inputs repeat after 251 rows, and so do the outputs, which a small call gives
    small, _, qs = moe.rms_norm(x[:251].clone(), gamma, 1e-6, q_scale=1 / 56)
    whole = T // 251
    assert (y[:whole * 251].view(whole, 251, H) == small).all() and (q[:whole * 251].view(whole, 251, H) == qs).all()
    assert torch.equal(y[whole * 251:], small[:T - whole * 251]) and torch.equal(q[whole * 251:], qs[:T - whole * 251])


def test_norm_refuses_one_place_for_two_outputs():
    dev = device()
    x, r, gamma = (t.to(dev) for t in _inputs(4, 64, torch.bfloat16, 1))
    for both in (x, r, torch.empty_like(x)):
        with pytest.raises(RuntimeError):
            moe.rms_norm(x, gamma, residual=r, y=both, residual_out=both)
    y, ro, _ = moe.rms_norm(x.clone(), gamma, residual=r.clone())
    got = moe.rms_norm(x, gamma, residual=r, y=x, residual_out=r)     # each in place of its own
    assert torch.equal(got[0], y) and torch.equal(got[1], ro)
