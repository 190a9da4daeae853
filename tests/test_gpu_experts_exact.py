"""The experts' gradients where they have to be exact, in the forms that only long or wide inputs take.

Inputs are small whole numbers, so that every product and every partial sum is a whole number under 2^24 in
size: f32 holds each of them, in whatever order they are added, and the results are compared bit for bit
with the same sums in 64 bits (a bf16 result with their one rounding). A row that is left out, taken twice or
read in another's place changes them.
"""
import pytest
import torch

import moe_expert_dispatch_amd as moe
from gpu_common import announce, device
from test_gpu_many_tokens import _free, _need

pytestmark = pytest.mark.gpu

B, F = torch.bfloat16, torch.float32


def _ints(g, most, *shape, dt=F):
    """Whole numbers from -most to most on the generator's device."""
    return torch.randint(-most, most + 1, shape, generator=g, device=g.device, dtype=torch.int8).to(dt)


def _gen(seed):
    return torch.Generator(device=device()).manual_seed(seed)


def _offsets(counts):
    return torch.cumsum(torch.tensor([0] + list(counts)), 0).to(torch.int32).to(device())


def _round(exact, dt):
    assert float(exact.abs().max()) < 2 ** 24
    return exact.to(F).to(dt)


def _weight_grad(dc, a, off):
    """[S, N, Kd] in 64 bits."""
    off = off.tolist()
    out = torch.zeros(len(off) - 1, dc.shape[1], a.shape[1], dtype=torch.float64, device=dc.device)
    for s, (lo, hi) in enumerate(zip(off, off[1:])):
        if hi > lo:
            out[s] = torch.mm(dc[lo:hi].double().t().contiguous(), a[lo:hi].double())
    return out


# bf16: 8, 4, 4 and 3 parts of 256 x 256 tiles; f32: 8 and 3 of 64 x 64. Slots without rows, of one slice, of
# three slices for four parts, and a part that ends inside a slice
SPLIT = [(B, [16384], 2048, 2048), (B, [12000, 0, 5, 4000], 2048, 1024), (B, [130, 8191, 64, 7000], 2048, 1024),
         (B, [9001, 7, 6993], 1800, 2056), (F, [6000], 512, 520), (F, [5000, 0, 130, 3000, 1], 328, 272)]


@pytest.mark.parametrize("dt,counts,N,Kd", SPLIT)
def test_split_rows_in_large_tiles(dt, counts, N, Kd):
    announce(f"split rows of large tiles {dt} {counts} N={N} Kd={Kd}")
    off, g = _offsets(counts), _gen(N + Kd)
    S, P = len(counts), sum(counts)
    assert moe.grouped_gemm_weight_grad_workspace_size(dt, S, P, N, Kd) >= 3 * S * N * Kd * 4
    dc, a = _ints(g, 2, P, N, dt=dt), _ints(g, 2, P, Kd, dt=dt)
    before = _ints(g, 100, S, N, Kd)
    exact = _weight_grad(dc, a, off)
    ws = torch.full((moe.grouped_gemm_weight_grad_workspace_size(dt, S, P, N, Kd),), 255, dtype=torch.uint8,
                    device=dc.device)  # NaNs in every part that is not written
    for odt in (F, B):
        for _ in range(2):
            assert torch.equal(moe.grouped_gemm_weight_grad(dc, a, off, dw_dtype=odt, ws=ws), _round(exact, odt)), odt
        dw = before.to(odt).clone()  # not before itself
        moe.grouped_gemm_weight_grad(dc, a, off, dw=dw, accumulate=True, ws=ws)
        assert torch.equal(dw, _round(exact + before.double(), odt)), f"{odt} accumulated"


@pytest.mark.parametrize("dt", [B, F])
def test_products_past_31_bits(dt):
    """Buffers of 70001 rows of 32768, the rows from 65536 on past 2^31 values: written by the rows' gradient, read
    by it and by the weights' gradient."""
    _need(60)
    rows, wide = 70001, 32768
    announce(f"exact gradients of {rows} rows of {wide} {dt}")
    g = _gen(6)
    off = torch.tensor([0, 100, 100, rows], dtype=torch.int32, device=g.device)
    slots = [(0, 0, 100), (2, 100, rows)]
    dc, w = _ints(g, 1, rows, 16, dt=dt), _ints(g, 1, 3, 16, wide, dt=dt)
    out = moe.grouped_gemm_backward(moe.DOWN, dc, off, w)
    for s, lo, hi in slots:
        for at in range(lo, hi, 4096):
            r = slice(at, min(at + 4096, hi))
            assert torch.equal(out[r], _round(torch.mm(dc[r].double(), w[s].double()), dt)), f"row {at} on"
    del dc, w
    # values of -1 to 1 in its place, for sums under 2^24
    for at in range(0, rows, 4096):
        out[at:at + 4096] = _ints(g, 1, *out[at:at + 4096].shape, dt=dt)
    back, a = _ints(g, 2, 3, wide, 8, dt=dt), _ints(g, 2, rows, 8, dt=dt)
    got = moe.grouped_gemm_backward(moe.DOWN, out, off, back)
    for s, lo, hi in slots:
        for at in range(lo, hi, 4096):
            r = slice(at, min(at + 4096, hi))
            assert torch.equal(got[r], _round(torch.mm(out[r].double(), back[s].double()), dt)), f"row {at} on, back"
    dw = moe.grouped_gemm_weight_grad(out, a, off)
    assert not dw[1].any()
    for s, lo, hi in slots:
        for c in range(0, wide, 4096):
            exact = torch.mm(out[lo:hi, c:c + 4096].double().t().contiguous(), a[lo:hi].double())
            assert torch.equal(dw[s, c:c + 4096], _round(exact, F)), f"slot {s}, column {c} on"
    del out, dw, got
    _free()
