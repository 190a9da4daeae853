"""SwiGLU and the gradients of the experts' products on the GPU against the fp64 oracle.

Tolerances, u = 2^-24. A product of n terms: bf16 products are exact, f32 ones round; each of at most n f32
additions of the matrix cores is within 2 u of its partial sum (whatever way it rounds), so the sum is within
2 n u + u of the terms' magnitudes. Then the output's rounding (bf16 2^-8, f32 u), with accumulate one more u
of the sum, with split rows at most 16 more.
The sigmoid: its argument's rounding |g| u 2, exp's and the quotient's few u, so 4 u (|g| + 4) relative; products
add one u each. The gradient's factor s + silu (1 - s) is at most 1.1 and at least -0.1: an error of
8 u (|g| + 4) s (1 + |g|).
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
TINY = 1e-40


def _offsets(counts):
    return torch.cumsum(torch.tensor([0] + list(counts)), 0).to(torch.int32)


COUNTS = {
    "one_row": [1],
    "empty_slots": [0, 3, 0, 0, 40, 0],
    "tile_ends": [256, 1, 255, 64, 63, 65, 128, 129],
    "two_tiles": [257, 0, 511],
    "many_slots": [(7 * i) % 5 for i in range(100)],
}


def _random(dt, seed, *shapes):
    g = torch.Generator().manual_seed(seed)
    return [torch.randn(*s, generator=g).to(dt) for s in shapes]


def _within(got, want, size, n, dt, what, more=0):
    err = (2 * n + 1 + more) * U * size
    assert_within(np64(got), want, err + ROUND[dt] * (np.abs(want) + err) + TINY, what)


@pytest.mark.parametrize("dt", [B, F])
@pytest.mark.parametrize("counts", list(COUNTS))
@pytest.mark.parametrize("Kd,N", [(8, 8), (64, 256), (72, 264), (200, 40), (520, 136)])
def test_rows_grad(dt, counts, Kd, N):
    """out[r] = dc[r] w[s] for both operations; rows behind the last slot's keep what they hold."""
    dev = device()
    announce(f"rows grad {dt} {counts} Kd={Kd} N={N}")
    off = _offsets(COUNTS[counts])
    S, P = len(off) - 1, int(off[-1])
    dc, w = _random(dt, Kd + N + P, (P + 5, Kd), (S, Kd, N))
    dc[P:] = float("nan")
    want = tr.grouped_rows_grad(dc[:P], off.numpy(), w)
    size = tr.grouped_rows_grad(dc[:P].abs(), off.numpy(), w.abs())
    ops = [moe.DOWN] + ([moe.GATE_UP_SWIGLU] if Kd % 16 == 0 else [])
    for op in ops:
        out = torch.full((P + 5, N), -7.0, device=dev).to(dt)
        got = moe.grouped_gemm_backward(op, dc.to(dev), off.to(dev), w.to(dev), out=out)
        assert got is out and (got[P:] == -7).all()
        _within(got[:P], want, size, Kd, dt, f"op {op}")


@pytest.mark.parametrize("dt", [B, F])
@pytest.mark.parametrize("counts", ["one_row", "empty_slots", "tile_ends"])
@pytest.mark.parametrize("H,I", [(8, 8), (64, 136), (136, 264), (72, 512)])
def test_swiglu_and_its_gradient(dt, counts, H, I):
    dev = device()
    announce(f"swiglu grad {dt} {counts} H={H} I={I}")
    off = _offsets(COUNTS[counts])
    S, P = len(off) - 1, int(off[-1])
    dy, w, h = _random(dt, H + I + P, (P + 3, H), (S, H, I), (P + 3, 2 * I))
    h = (h.float() * 4).to(dt)
    h[0, :4] = torch.tensor([-60.0, 60.0, 0.0, -1.2785])
    h[P:] = float("nan")
    hd = np64(h[:P])
    g, u = hd[:, :I], hd[:, I:]
    s = tr.sigmoid(g)
    act = moe.swiglu(h.to(dev), off.to(dev), act=torch.full((P + 3, I), -7.0, device=dev).to(dt))
    assert (act[P:] == -7).all()
    want = tr.swiglu(h[:P])
    err = 4 * U * (np.abs(g) + 6) * np.abs(want)
    assert_within(np64(act[:P]), want, err + ROUND[dt] * (np.abs(want) + err) + TINY, "act")
    out = torch.full((P + 3, 2 * I), -7.0, device=dev).to(dt)
    dh = moe.grouped_gemm_backward(moe.DOWN, dy.to(dev), off.to(dev), w.to(dev), h=h.to(dev), out=out)
    assert (dh[P:] == -7).all()
    da = tr.grouped_rows_grad(dy[:P], off.numpy(), w)
    da_err = (2 * H + 1) * U * tr.grouped_rows_grad(dy[:P].abs(), off.numpy(), w.abs())
    want = tr.swiglu_backward(h[:P], da)
    slope = np.concatenate([np.abs(u * s * (1 + g * (1 - s))), np.abs(g * s)], 1)
    rest = np.concatenate([np.abs(u) * s * (1 + np.abs(g)), np.abs(g) * s], 1)
    da2, de2 = np.tile(np.abs(da), (1, 2)), np.tile(da_err, (1, 2))
    ga = np.tile(np.abs(g), (1, 2))
    err = de2 * (slope + 8 * U * (ga + 6) * rest) + da2 * 8 * U * (ga + 6) * rest
    assert_within(np64(dh[:P]), want, err + ROUND[dt] * (np.abs(want) + err) + TINY, "dh")


@pytest.mark.parametrize("dt", [B, F])
@pytest.mark.parametrize("counts", list(COUNTS))
@pytest.mark.parametrize("N,Kd", [(8, 8), (256, 64), (264, 72), (40, 200), (136, 520)])
def test_weight_grad(dt, counts, N, Kd):
    dev = device()
    announce(f"weight grad {dt} {counts} N={N} Kd={Kd}")
    off = _offsets(COUNTS[counts])
    S, P = len(off) - 1, int(off[-1])
    dc, a, before = _random(dt, N + Kd + P, (P + 5, N), (P + 5, Kd), (S, N, Kd))
    dc[P:] = float("nan")
    a[P:] = float("inf")
    want = tr.grouped_weight_grad(dc[:P], a[:P], off.numpy())
    size = tr.grouped_weight_grad(dc[:P].abs(), a[:P].abs(), off.numpy())
    n = int(max(COUNTS[counts]))
    for odt in (F, B):
        got = moe.grouped_gemm_weight_grad(dc.to(dev), a.to(dev), off.to(dev), dw_dtype=odt)
        _within(got, want, size, n, odt, f"{odt}")
        start = before.to(odt)
        dw = start.to(dev)
        got = moe.grouped_gemm_weight_grad(dc.to(dev), a.to(dev), off.to(dev), dw=dw, accumulate=True)
        assert got is dw
        total = want + np64(start)
        _within(got, total, size + np.abs(total), n, odt, f"{odt} accumulated")
        for s in range(S):
            if off[s] == off[s + 1]:
                assert torch.equal(dw[s].cpu(), start[s])


@pytest.mark.parametrize("dt", [B, F])
@pytest.mark.parametrize("counts,N,Kd", [([9000], 64, 40), ([0, 4000, 3], 264, 72), ([3000, 1, 0, 2999], 16, 136)])
def test_split_rows(dt, counts, N, Kd):
    """Few tiles and many rows: the parts add up, also where a split gets no rows; runs repeat bit for bit."""
    dev = device()
    announce(f"split rows {dt} {counts} N={N} Kd={Kd}")
    off = _offsets(counts)
    S, P = len(off) - 1, int(off[-1])
    assert moe.grouped_gemm_weight_grad_workspace_size(dt, S, P, N, Kd) > 0
    dc, a, before = _random(dt, P, (P, N), (P, Kd), (S, N, Kd))
    want = tr.grouped_weight_grad(dc, a, off.numpy())
    size = tr.grouped_weight_grad(dc.abs(), a.abs(), off.numpy())
    for odt in (F, B):
        D, A, O = dc.to(dev), a.to(dev), off.to(dev)
        got = moe.grouped_gemm_weight_grad(D, A, O, dw_dtype=odt)
        _within(got, want, size, max(counts), odt, f"{odt}", more=16)
        for _ in range(3):
            assert torch.equal(moe.grouped_gemm_weight_grad(D, A, O, dw_dtype=odt), got)
        dw = before.to(odt).to(dev)
        moe.grouped_gemm_weight_grad(D, A, O, dw=dw, accumulate=True)
        total = want + np64(before.to(odt))
        _within(dw, total, size + np.abs(total), max(counts), odt, f"{odt} accumulated", more=16)


def test_wide_and_long():
    """Several column tiles, contractions of many slices, a long slot beside short ones."""
    dev = device()
    for dt, counts, H, I in ((B, [700, 0, 5, 300], 1032, 520), (B, [130, 70], 2048, 1408), (F, [200, 3], 520, 264)):
        announce(f"wide {dt} {counts} {H} {I}")
        off = _offsets(counts)
        S, P = len(off) - 1, int(off[-1])
        dy, w, a = _random(dt, H, (P, H), (S, H, I), (P, I))
        got = moe.grouped_gemm_backward(moe.DOWN, dy.to(dev), off.to(dev), w.to(dev))
        _within(got, tr.grouped_rows_grad(dy, off.numpy(), w), tr.grouped_rows_grad(dy.abs(), off.numpy(), w.abs()), H, dt, "rows")
        got = moe.grouped_gemm_weight_grad(dy.to(dev), a.to(dev), off.to(dev))
        _within(got, tr.grouped_weight_grad(dy, a, off.numpy()), tr.grouped_weight_grad(dy.abs(), a.abs(), off.numpy()),
                max(counts), F, "weights")


def test_no_rows():
    dev = device()
    off = torch.zeros(4, dtype=torch.int32, device=dev)
    dc, a, w = torch.empty(0, 64, device=dev), torch.empty(0, 40, device=dev), torch.randn(3, 64, 40, device=dev)
    for dt in (B, F):
        dw = torch.full((3, 64, 40), 3.0, device=dev)
        moe.grouped_gemm_weight_grad(dc.to(dt), a.to(dt), off, dw=dw)
        assert not dw.any()
        assert moe.grouped_gemm_backward(moe.DOWN, dc.to(dt), off, w.to(dt)).shape == (0, 40)
        # rows there, but none in a slot
        full = torch.full((9, 40), 2.0, device=dev).to(dt)
        moe.grouped_gemm_backward(moe.DOWN, torch.randn(9, 64, device=dev).to(dt), off, w.to(dt), out=full)
        assert (full == 2).all()


def test_values_stay_in_their_row_and_slot():
    """A NaN or an infinity of one row reaches its own gradient row and its own slot's weights only."""
    dev = device()
    off = _offsets([70, 5, 61]).to(dev)
    for dt in (B, F):
        dc, w, a = (t.to(dev) for t in _random(dt, 5, (136, 72), (3, 72, 40), (136, 40)))
        rows, weights = moe.grouped_gemm_backward(moe.DOWN, dc, off, w), moe.grouped_gemm_weight_grad(dc, a, off)
        dc[69, 71], dc[75, 0], w[1, 3, 3] = float("nan"), float("inf"), float("nan")
        r2, w2 = moe.grouped_gemm_backward(moe.DOWN, dc, off, w), moe.grouped_gemm_weight_grad(dc, a, off)
        keep = [i for i in range(136) if i not in (69, 75) and not 70 <= i < 75]
        assert torch.equal(r2[keep], rows[keep])
        assert torch.equal(w2[1], weights[1]) and torch.equal(w2[0, :71], weights[0, :71])
        assert torch.equal(w2[2, 1:], weights[2, 1:]) and not torch.isfinite(w2[2, 0]).any()


def test_offsets_past_the_rows():
    """Offsets that claim more rows than the buffers hold touch nothing behind them."""
    dev = device()
    off = torch.tensor([0, 6, 400, 900], dtype=torch.int32, device=dev)
    for dt in (B, F):
        dc, w, a, h = (t.to(dev) for t in _random(dt, 6, (16, 64), (3, 64, 40), (16, 40), (16, 80)))
        cut = torch.tensor([0, 6, 16, 16], dtype=torch.int32, device=dev)
        for one, two in ((moe.grouped_gemm_backward(moe.DOWN, dc, off, w), moe.grouped_gemm_backward(moe.DOWN, dc, cut, w)),
                         (moe.grouped_gemm_weight_grad(dc, a, off), moe.grouped_gemm_weight_grad(dc, a, cut)),
                         (moe.swiglu(h, off), moe.swiglu(h, cut))):
            assert torch.equal(one, two)


def test_refusals():
    dev = device()
    off = _offsets([3, 5]).to(dev)
    dc, w, a, h = (t.to(dev) for t in _random(F, 7, (8, 64), (2, 64, 40), (8, 40), (8, 80)))
    for bad in (lambda: moe.grouped_gemm_backward(moe.DOWN, dc, off, w.bfloat16()),
                lambda: moe.grouped_gemm_backward(moe.DOWN, dc, off, w, h=h.bfloat16()),
                lambda: moe.grouped_gemm_backward(moe.DOWN, dc.half(), off, w.half()),
                lambda: moe.grouped_gemm_weight_grad(dc, a.bfloat16(), off),
                lambda: moe.grouped_gemm_weight_grad(dc, a, off, dw_dtype=torch.float16),
                lambda: moe.swiglu(h.half(), off), lambda: moe.swiglu(h, off.long())):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: moe.grouped_gemm_backward(moe.DOWN, dc, off[:2], w), lambda: moe.grouped_gemm_backward(2, dc, off, w),
                lambda: moe.grouped_gemm_backward(moe.GATE_UP_SWIGLU, dc, off, w, h=h),
                lambda: moe.grouped_gemm_backward(moe.DOWN, dc[:, :32], off, w),
                lambda: moe.grouped_gemm_backward(moe.DOWN, dc, off, w, h=h[:, :40]),
                lambda: moe.grouped_gemm_weight_grad(dc, a[:4], off),
                lambda: moe.grouped_gemm_weight_grad(dc, a, off, accumulate=True),
                lambda: moe.grouped_gemm_weight_grad(dc, a.cpu(), off), lambda: moe.swiglu(h[:, :79], off),
                lambda: moe.swiglu(h, off, act=torch.empty(8, 80, device=dev))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(RuntimeError):
        moe.swiglu(torch.zeros(8, 24, device=dev), off)   # 2I of a half that is no multiple of 8


# every way that a tile of 256 (or 64) rows ends, in enough tiles that the large ones are taken
ENDS = [0, 1, 31, 32, 33, 63, 64, 65, 95, 97, 127, 128, 129, 160, 191, 192, 193, 223, 224, 225, 255, 256, 257, 300, 384,
        511, 512, 513]


@pytest.mark.parametrize("dt", [B, F])
@pytest.mark.parametrize("Kd", [8, 64, 72, 128, 200, 264])
def test_large_tiles_of_rows(dt, Kd):
    dev = device()
    N = 1032
    announce(f"large tiles rows {dt} Kd={Kd}")
    off = _offsets(ENDS)
    S, P = len(off) - 1, int(off[-1])
    dc, w, h = _random(dt, Kd, (P + 9, Kd), (S, Kd, N), (P + 9, 2 * N))
    dc[P:] = float("nan")
    h[P:] = float("nan")
    args = (moe.DOWN, dc.to(dev), off.to(dev), w.to(dev))
    want = tr.grouped_rows_grad(dc[:P], off.numpy(), w)
    size = tr.grouped_rows_grad(dc[:P].abs(), off.numpy(), w.abs())
    for again in range(3):  # many tiles a block, one after the other: the same bits each time
        out = torch.full((P + 9, N), -7.0, device=dev).to(dt)
        got = moe.grouped_gemm_backward(*args, out=out)
        assert (got[P:] == -7).all()
        if again:
            assert torch.equal(got, first)
        first = got
    _within(got[:P], want, size, Kd, dt, "rows")
    dh = moe.grouped_gemm_backward(*args, h=h.to(dev), out=torch.full((P + 9, 2 * N), -7.0, device=dev).to(dt))
    assert (dh[P:] == -7).all()
    hd = np64(h[:P])
    g, u = hd[:, :N], hd[:, N:]
    s = tr.sigmoid(g)
    want2 = tr.swiglu_backward(h[:P], want)
    slope = np.concatenate([np.abs(u * s * (1 + g * (1 - s))), np.abs(g * s)], 1)
    rest = np.concatenate([np.abs(u) * s * (1 + np.abs(g)), np.abs(g) * s], 1)
    da, de, ga = (np.tile(a, (1, 2)) for a in (np.abs(want), (2 * Kd + 1) * U * size, np.abs(g)))
    err = de * (slope + 8 * U * (ga + 6) * rest) + da * 8 * U * (ga + 6) * rest
    assert_within(np64(dh[:P]), want2, err + ROUND[dt] * (np.abs(want2) + err) + TINY, "dh")


@pytest.mark.parametrize("dt", [B, F])
@pytest.mark.parametrize("N,Kd", [(264, 520), (520, 264), (1032, 72), (1032, 520), (520, 1288)])
def test_many_tiles_of_weights(dt, N, Kd):
    dev = device()
    announce(f"many tiles weights {dt} N={N} Kd={Kd}")
    off = _offsets(ENDS)
    S, P = len(off) - 1, int(off[-1])
    dc, a, before = _random(dt, N, (P + 9, N), (P + 9, Kd), (S, N, Kd))
    dc[P:] = float("nan")
    want = tr.grouped_weight_grad(dc[:P], a[:P], off.numpy())
    size = tr.grouped_weight_grad(dc[:P].abs(), a[:P].abs(), off.numpy())
    D, A, O = dc.to(dev), a.to(dev), off.to(dev)
    for odt in (F, B):
        first = moe.grouped_gemm_weight_grad(D, A, O, dw_dtype=odt)
        _within(first, want, size, max(ENDS), odt, f"{odt}")
        for _ in range(3):
            assert torch.equal(moe.grouped_gemm_weight_grad(D, A, O, dw_dtype=odt), first)
        dw = before.to(odt).to(dev)
        moe.grouped_gemm_weight_grad(D, A, O, dw=dw, accumulate=True)
        total = want + np64(before.to(odt))
        _within(dw, total, size + np.abs(total), max(ENDS), odt, f"{odt} accumulated")


@pytest.mark.parametrize("dt", [B, F])
def test_the_most_slots(dt):
    dev = device()
    announce(f"1024 slots {dt}")
    counts = [(5 * i) % 7 for i in range(1024)]
    off = _offsets(counts)
    S, P = 1024, int(off[-1])
    dc, w, a = _random(dt, 3, (P, 40), (S, 40, 24), (P, 24))
    got = moe.grouped_gemm_backward(moe.DOWN, dc.to(dev), off.to(dev), w.to(dev))
    _within(got, tr.grouped_rows_grad(dc, off.numpy(), w), tr.grouped_rows_grad(dc.abs(), off.numpy(), w.abs()), 40, dt, "rows")
    got = moe.grouped_gemm_weight_grad(dc.to(dev), a.to(dev), off.to(dev))
    _within(got, tr.grouped_weight_grad(dc, a, off.numpy()), tr.grouped_weight_grad(dc.abs(), a.abs(), off.numpy()), 7, F, "weights")


@pytest.mark.parametrize("dt", [B, F])
def test_rows_before_the_first_slot(dt):
    """Slots that begin behind row 0: the rows before them are left as they were, whatever they hold."""
    dev = device()
    announce(f"rows before the first slot {dt}")
    off = torch.tensor([37, 37, 90, 111], dtype=torch.int32)
    dc, w, a, h = _random(dt, 7, (130, 72), (3, 72, 40), (130, 40), (130, 80))
    for t in (dc, a, h):
        t[:37] = float("nan")
        t[111:] = float("nan")
    D, W, A, H, O = (t.to(dev) for t in (dc, w, a, h, off))
    inner = lambda t: t[37:111].contiguous()  # noqa: E731
    O0 = O - 37
    blank = lambda n: torch.full((130, n), -7.0, device=dev).to(dt)  # noqa: E731
    for got, want in ((moe.swiglu(H, O, act=blank(40)), moe.swiglu(inner(H), O0)),
                      (moe.grouped_gemm_backward(moe.DOWN, D, O, W, out=blank(40)),
                       moe.grouped_gemm_backward(moe.DOWN, inner(D), O0, W)),
                      (moe.grouped_gemm_backward(moe.DOWN, D, O, W, h=H, out=blank(80)),
                       moe.grouped_gemm_backward(moe.DOWN, inner(D), O0, W, h=inner(H)))):
        assert torch.equal(got[37:111], want) and torch.isfinite(want).all()
        assert (got[:37] == -7).all() and (got[111:] == -7).all()
    assert torch.equal(moe.grouped_gemm_weight_grad(D, A, O), moe.grouped_gemm_weight_grad(inner(D), inner(A), O0))


def test_workspaces_are_contiguous():
    """A workspace that holds one byte over and over has the bytes that are asked for, but not the memory."""
    dev = device()
    one = torch.zeros(1, dtype=torch.uint8, device=dev).expand(1 << 24)
    x, off = torch.zeros(400, 64, device=dev), _offsets([400]).to(dev)
    for bad in (lambda: moe.grouped_gemm_weight_grad(x, x, off, ws=one),
                lambda: moe.layer_norm_backward(x, x, x[0], ws=one), lambda: moe.rms_norm_backward(x, x, x[0], ws=one)):
        with pytest.raises(ValueError):
            bad()
