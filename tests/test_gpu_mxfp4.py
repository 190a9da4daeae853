"""MXFP4 expert weights on the GPU against the fp64 oracle.

Quantisation and its inverse are compared bit for bit. In the products every
term is exact (a code times its scale has two significant bits, the
activation eight), so a sum of Kd terms in f32, in any order, is within
Kd u sum|terms| of the exact one, u = 2^-24 (MFMA sums may truncate: twice
that is allowed). The SwiGLU carries those bounds (|silu'| < 1.1), with 16 u
for its own evaluation, and rounds once to bf16 (2^-8). A layer's output
carries the rounding of the bf16 activations, 2^-8 of the magnitudes they
are weighted with, the sums, and its own rounding.
"""
import numpy as np
import pytest
import torch

import moe_expert_dispatch_amd as moe
import oracle
from gpu_common import announce, device, np64
from workloads import build_slot_table

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def _weights(shape, seed, fan):
    """Quantised Gaussian weights, groups of several widths: (codes, scales)."""
    g = np.random.default_rng(seed)
    w = g.standard_normal(shape) / np.sqrt(fan) * np.repeat(
        2.0 ** g.integers(-2, 3, (*shape[:-1], shape[-1] // 32)), 32, axis=-1)
    c, s = oracle.mxfp4_encode(w)
    return torch.from_numpy(c), torch.from_numpy(s)


def _rows(n, k, seed):
    return torch.randn(n, k, generator=torch.Generator().manual_seed(seed)).bfloat16()


# ------------------------------------------------------------------ weights
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape", [(32,), (1, 64), (3, 5, 96), (7, 2048), (129, 4128)])
def test_quantize_bit_exact(dt, shape):
    dev = device()
    announce(f"quantize mxfp4 {dt} {shape}")
    g = torch.Generator().manual_seed(sum(shape))
    w = torch.randn(shape, generator=g) * 10.0 ** torch.randint(-6, 6, shape, generator=g).float()
    flat = w.view(-1, 32)
    flat[0] = torch.tensor([6.0, .25, .75, 1.25, 1.75, 2.5, 3.5, 5.0] * 4)
    flat[0, 8:16] *= -1
    if flat.shape[0] > 4:
        flat[1] = 0.0
        flat[2] *= 1e-42                        # subnormal values
        flat[3, 3] = float("inf")
        flat[4, 31] = float("nan")
    w = w.to(dt)
    codes, scale = moe.quantize_mxfp4(w.to(dev))
    want_c, want_s = oracle.mxfp4_encode(w)
    assert np.array_equal(scale.cpu().numpy(), want_s)
    fine = np.repeat(want_s != 255, 16, axis=-1)  # the codes of a NaN group are unspecified
    assert np.array_equal(codes.cpu().numpy()[fine], want_c[fine])
    for out in (torch.bfloat16, torch.float32):
        v = moe.dequantize_mxfp4(codes, scale, out)
        want = torch.from_numpy(oracle.mxfp4_decode(codes, scale)).to(out)
        assert torch.equal(torch.nan_to_num(v.cpu(), nan=12345.0), torch.nan_to_num(want, nan=12345.0))


def test_dequantize_every_code_and_scale():
    dev = device()
    announce("dequantize every byte and scale")
    codes = torch.arange(256, dtype=torch.uint8).repeat(256, 1)          # 16 groups a row
    scale = torch.arange(256, dtype=torch.uint8)[:, None].repeat(1, 16)
    for dt in (torch.bfloat16, torch.float32):
        v = moe.dequantize_mxfp4(codes.to(dev), scale.to(dev), dt).cpu()
        want = torch.from_numpy(oracle.mxfp4_decode(codes, scale)).to(dt)
        assert torch.equal(torch.nan_to_num(v, nan=12345.0, posinf=9e30, neginf=-9e30),
                           torch.nan_to_num(want, nan=12345.0, posinf=9e30, neginf=-9e30)), dt


def test_quantize_empty_and_refusals():
    dev = device()
    c, s = moe.quantize_mxfp4(torch.empty(0, 64, device=dev))
    assert c.shape == (0, 32) and s.shape == (0, 2)
    assert moe.dequantize_mxfp4(c, s).shape == (0, 64)
    with pytest.raises(ValueError):
        moe.quantize_mxfp4(torch.zeros(4, 48, device=dev))
    with pytest.raises(TypeError):
        moe.quantize_mxfp4(torch.zeros(4, 64, device=dev, dtype=torch.float16))
    with pytest.raises(ValueError):
        moe.dequantize_mxfp4(torch.zeros(4, 32, device=dev, dtype=torch.uint8),
                             torch.zeros(4, 4, device=dev, dtype=torch.uint8))
    with pytest.raises(TypeError):
        moe.dequantize_mxfp4(torch.zeros(4, 16, device=dev, dtype=torch.uint8),
                             torch.zeros(4, 1, device=dev, dtype=torch.uint8), torch.float16)


def test_quantize_more_groups_than_a_grid_line_has_threads_for():
    """2^35 + 96 weights, four threads a group: past the 2^32 threads of one grid dimension. The weights repeat
    every 4128 groups, and so have to the codes, the scales and the weights read back."""
    dev = device()
    announce("quantize mxfp4 2^35 + 96")
    n, period = 2 ** 35 + 96, 4128 * 32
    if torch.cuda.mem_get_info()[0] < 100 * 2 ** 30:
        pytest.skip("needs 100 GiB of device memory")
    g = torch.Generator(device=dev).manual_seed(4)
    part = torch.randn(period, generator=g, device=dev) * torch.randn(period // 32, generator=g, device=dev).exp(
    ).repeat_interleave(32)
    part = part.bfloat16()
    whole = n // period
    w = torch.empty(n, dtype=torch.bfloat16, device=dev)
    w[:whole * period].view(whole, period).copy_(part.expand(whole, period))
    w[whole * period:] = part[:n - whole * period]
    codes, scale = moe.quantize_mxfp4(w)
    pc, ps = moe.quantize_mxfp4(part)
    pw = moe.dequantize_mxfp4(pc, ps)

    def repeats(t, one):
        m = one.numel()
        lines, left = t[:whole * m].view(whole, m), t[whole * m:]
        step = 1 << 14                       # a few GB of truth values at a time
        return all(bool((lines[i:i + step] == one).all()) for i in range(0, whole, step)) and torch.equal(
            left, one[:left.numel()])
    assert repeats(codes, pc) and repeats(scale, ps)
    w.zero_()
    moe.dequantize_mxfp4(codes, scale, out=w)
    assert repeats(w, pw)
    del w, codes, scale
    torch.cuda.empty_cache()


# ------------------------------------------------------------------ products
SIZES = [[1], [0, 1, 0], [3, 0, 16, 1], [17, 0, 5, 33], [70, 1, 0, 0, 2], [300, 129], [0, 0],
         [40, 64, 65, 8, 9, 4, 5, 2],
         # enough rows a slot for the tiles of 128, with every number of 32-row blocks in one
         [0, 500, 0, 31, 97, 128, 0, 0, 4, 0], [33], [64, 1], [96, 160, 129, 0], [0] * 70 + [4000, 1, 0]]


def _offsets(sizes):
    return torch.tensor(np.concatenate([[0], np.cumsum(sizes)]), dtype=torch.int32)


def _products_check(sizes, H, I):
    dev = device()
    announce(f"mxfp4 products {sizes} H={H} I={I}")
    S, rows, off = len(sizes), int(sum(sizes)), _offsets(sizes)
    gu, gs = _weights((S, 2 * I, H), H + I, H)
    wd, ds = _weights((S, H, I), H * 3 + I, I)
    x = _rows(rows, H, rows + H)
    act = moe.grouped_gemm_mxfp4(moe.GATE_UP_SWIGLU, x.to(dev), off.to(dev), gu.to(dev), gs.to(dev))
    want, g, u, gm, um = oracle.mxfp4_grouped_gate_up(x, off, gu, gs, I)
    dg, du = 2 * H * U * gm, 2 * H * U * um
    tol = (1.1 * dg * (np.abs(u) + du) + np.abs(oracle.silu(g)) * du + (2.0 ** -8 + 16 * U) * np.abs(want)) * 1.01
    assert (np.abs(np64(act) - want) <= tol + 1e-38).all()
    y = moe.grouped_gemm_mxfp4(moe.DOWN, act, off.to(dev), wd.to(dev), ds.to(dev), c_dtype=torch.float32)
    want, m = oracle.mxfp4_grouped_down(act.cpu(), off, wd, ds)
    assert (np.abs(np64(y) - want) <= (2 * I * U * m + 2 * U * np.abs(want)) * 1.01 + 1e-38).all()


# every way the products are split: rows a slot (up to 2, 4, 10, 24, 56 and more on the average, with
# slots far over and under it) by short, middle and long contractions and ones that are no multiple of 128
ROWS = {"two": [2, 0, 1, 9, 0, 2] * 4, "four": [4, 0, 9, 3], "ten": [0, 10, 17, 13], "twenty": [33, 0, 40, 7],
        "fifty": [65, 50, 0, 70], "hundred": [1, 300, 0, 96],
        # tiles of 160: one, one row past it, two of one size, three, and every number of 32s in the last
        "tiles": [160, 161, 320, 321, 0, 130, 481, 641]}


@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("H,I", [(96, 1056), (384, 640), (1152, 160), (2176, 64), (3968, 32), (4096, 32), (4128, 32),
                                 (8320, 32), (9248, 32)])
def test_products_every_split(rows, H, I):
    _products_check(ROWS[rows], H, I)


@pytest.mark.parametrize("rows", [[160, 161, 320, 321, 0, 130, 481, 1727], [33, 2900, 0, 400]])
@pytest.mark.parametrize("H,I", [(1120, 672), (2176, 640), (32, 2720), (1120, 320), (2176, 320)])
def test_products_in_large_tiles(rows, H, I):
    """As many rows and columns as fill the chip with the largest tiles, or (320 columns) the middle ones, over
    whole and broken steps."""
    _products_check(rows, H, I)


@pytest.mark.parametrize("sizes", SIZES, ids=str)
@pytest.mark.parametrize("H,I", [(32, 32), (64, 96), (160, 32), (512, 224), (1024, 128), (2048, 64)])
def test_products_against_oracle(sizes, H, I):
    dev = device()
    announce(f"mxfp4 products {sizes} H={H} I={I}")
    S, rows, off = len(sizes), int(sum(sizes)), _offsets(sizes)
    cap = rows + 5                             # rows behind the last slot stay as they are
    gu, gs = _weights((S, 2 * I, H), H + I, H)
    wd, ds = _weights((S, H, I), H * 3 + I, I)
    x = _rows(cap, H, rows + H)
    act = torch.full((cap, I), -77.0, dtype=torch.bfloat16, device=dev)
    moe.grouped_gemm_mxfp4(moe.GATE_UP_SWIGLU, x.to(dev), off.to(dev), gu.to(dev), gs.to(dev), act)
    want, g, u, gm, um = oracle.mxfp4_grouped_gate_up(x[:rows], off, gu, gs, I)
    dg, du = 2 * H * U * gm, 2 * H * U * um
    sl = np.abs(oracle.silu(g))
    tol = 1.1 * dg * (np.abs(u) + du) + sl * du + (2.0 ** -8 + 16 * U) * np.abs(want) + 1e-38
    got = np64(act)
    assert (np.abs(got[:rows] - want) <= tol * 1.01).all()
    assert (got[rows:] == -77.0).all()
    a2 = act[:, :].clone()
    a2[rows:] = float("nan")
    for dt, r in ((torch.bfloat16, 2.0 ** -8), (torch.float32, 2 * U)):
        y = torch.full((cap, H), -77.0, dtype=dt, device=dev)
        moe.grouped_gemm_mxfp4(moe.DOWN, a2, off.to(dev), wd.to(dev), ds.to(dev), y)
        want, m = oracle.mxfp4_grouped_down(a2[:rows].cpu(), off, wd, ds)
        got = np64(y)
        assert (np.abs(got[:rows] - want) <= (2 * I * U * m + r * np.abs(want)) * 1.01 + 1e-38).all()
        assert (got[rows:] == -77.0).all()


def test_products_with_nan_scale_and_capacity():
    """A weight with scale 255 makes its own column NaN and no other; rows past the capacity that
    offsets claim are not touched."""
    dev = device()
    announce("mxfp4 products, NaN scale")
    H, I = 128, 64
    wd, ds = _weights((2, H, I), 3, I)
    ds[1, 5, 1] = 255
    a = _rows(12, I, 1)
    off = torch.tensor([0, 4, 12], dtype=torch.int32)
    y = moe.grouped_gemm_mxfp4(moe.DOWN, a.to(dev), off.to(dev), wd.to(dev), ds.to(dev),
                               c_dtype=torch.float32).cpu()
    nan = torch.isnan(y)
    assert nan[4:, 5].all() and int(nan.sum()) == 8
    c = torch.full((12, H), 3.0, device=dev)
    so = moe.lib()
    ad, od, wdd, dsd = (t.to(dev) for t in (a, off, wd, ds))
    assert so.moe_grouped_gemm_mxfp4(1, ad.data_ptr(), od.data_ptr(), 2, 6, wdd.data_ptr(), dsd.data_ptr(),
                                     H, I, c.data_ptr(), 0, torch.cuda.current_stream().cuda_stream) == 0
    assert (c[6:] == 3.0).all() and torch.equal(c[:4].cpu(), y[:4])


@pytest.mark.parametrize("low", [0, 246])
@pytest.mark.parametrize("rows", [1, 3, 9, 20, 60, 200])
def test_products_at_the_ends_of_the_scales(low, rows):
    """The least scales (weights below bf16's normal numbers) with large activations, and the largest with small
    ones: products are exact there too."""
    dev = device()
    announce(f"mxfp4 products scales from {low} rows={rows}")
    H, I, S = 256, 160, 2
    g = torch.Generator().manual_seed(low + rows)
    wd = torch.randint(0, 256, (S, H, I // 2), generator=g, dtype=torch.uint8)
    ds = torch.randint(low, low + 7, (S, H, I // 32), generator=g, dtype=torch.uint8)
    a = (torch.randn(S * rows, I, generator=g) * (2.0 ** 110 if low == 0 else 2.0 ** -110)).bfloat16()
    off = _offsets([rows] * S)
    y = moe.grouped_gemm_mxfp4(moe.DOWN, a.to(dev), off.to(dev), wd.to(dev), ds.to(dev), c_dtype=torch.float32)
    want, m = oracle.mxfp4_grouped_down(a, off, wd, ds)
    assert (np.abs(np64(y) - want) <= (2 * I * U * m + 2 * U * np.abs(want)) * 1.01).all()


def test_products_refusals():
    dev = device()
    w, s = _weights((2, 64, 64), 1, 64)
    w, s, off, a = w.to(dev), s.to(dev), _offsets([1, 2]).to(dev), _rows(3, 64, 1).to(dev)
    for bad in (lambda: moe.grouped_gemm_mxfp4(0, a.float(), off, w, s),
                lambda: moe.grouped_gemm_mxfp4(0, a, off, w, s.int()),
                lambda: moe.grouped_gemm_mxfp4(0, a, off, w, s, c_dtype=torch.float32)):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: moe.grouped_gemm_mxfp4(0, a, off[:2], w, s),
                lambda: moe.grouped_gemm_mxfp4(0, a[:, :32].contiguous(), off, w, s),
                lambda: moe.grouped_gemm_mxfp4(2, a, off, w, s),
                lambda: moe.grouped_gemm_mxfp4(0, a, off, w, s[:, :, :1].contiguous())):
        with pytest.raises(ValueError):
            bad()


# ------------------------------------------------------------------ layer
def _layer(T, H, I, E, K, seed, ep=1, extra=0, skew=0.0):
    El = E // ep
    gu, gs = _weights((E, 2 * I, H), seed, H)
    wd, ds = _weights((E, H, I), seed + 1, I)
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, H, generator=g).bfloat16()
    logits = torch.randn(T, E, generator=g) + skew * torch.randn(E, generator=g)
    ro, rs, se = build_slot_table(El, list(range(extra)))
    return dict(gu=gu, gs=gs, wd=wd, ds=ds, x=x, logits=logits, ro=ro, rs=rs, se=se.long(), El=El,
                cfg=dict(H=H, I=I, E_global=E, K=K, renormalize=True, S=El + extra, dtype=moe.MXFP4,
                         ep_size=ep))


def _run(dev, L, T, rank=0, **kw):
    lo = rank * L["El"]
    at = lo + L["se"]
    cfg = moe.ForwardConfig(T=T, ep_rank=rank, **{**L["cfg"], **kw.pop("cfg", {})})
    put = {k: (v.to(dev) if isinstance(v, torch.Tensor) else v) for k, v in kw.items()}
    return moe.forward(cfg, L["x"][:T].to(dev), L["gu"][at].to(dev), L["wd"][at].to(dev),
                       rep_off=L["ro"].to(dev), rep_slots=L["rs"].to(dev),
                       w_gate_up_scale=L["gs"][at].to(dev), w_down_scale=L["ds"][at].to(dev), **put)


def _reference(L, T, ids, w, rank=0, on_input=False):
    """(output, allowance): the layer in 64 bits over (ids, w), and what the roundings may move it."""
    El, H, I = L["El"], L["cfg"]["H"], L["cfg"]["I"]
    out, tol = np.zeros((T, H)), np.zeros((T, H))
    x = np64(L["x"])
    for e in range(rank * El, (rank + 1) * El):
        t, k = np.nonzero(ids[:T] == e)
        if not t.size:
            continue
        wt = w[t, k][:, None]
        xin = x[t]
        if on_input:
            xin = (L["x"][t].float() * torch.from_numpy(wt).float()).bfloat16().double().numpy()
            wt = np.ones_like(wt)
        off = np.array([0, t.size])
        a, g, u, gm, um = oracle.mxfp4_grouped_gate_up(xin, off, L["gu"][e:e + 1], L["gs"][e:e + 1], I)
        y, m = oracle.mxfp4_grouped_down(a, off, L["wd"][e:e + 1], L["ds"][e:e + 1])
        dg, du = 2 * H * U * gm, 2 * H * U * um
        da = 1.1 * dg * (np.abs(u) + du) + np.abs(oracle.silu(g)) * du + (2.0 ** -8 + 16 * U) * np.abs(a)
        dwn = np.abs(oracle.mxfp4_decode(L["wd"][e], L["ds"][e]))
        out[t] += wt * y
        tol[t] += wt * (da @ dwn.T * 1.01 + (2 * I + 64) * U * m)
    return out, tol


LAYERS = {
    "one_token": dict(T=1, H=256, I=96, E=8, K=2, seed=1),
    "one_token_ep": dict(T=1, H=512, I=64, E=16, K=4, seed=2, ep=4),
    "two_tokens": dict(T=2, H=4224, I=608, E=12, K=5, seed=10, ep=2, extra=2),
    "two_odd": dict(T=2, H=160, I=96, E=6, K=6, seed=11, extra=1),
    "long_rows": dict(T=3, H=5216, I=1056, E=3, K=2, seed=12),
    "plan_limit": dict(T=128, H=64, I=32, E=24, K=8, seed=13, extra=5),
    "past_plan": dict(T=129, H=64, I=32, E=24, K=8, seed=14, ep=2),
    "many_experts": dict(T=6, H=64, I=32, E=512, K=6, seed=15),
    "most_slots": dict(T=128, H=32, I=32, E=1024, K=8, seed=16),
    "few": dict(T=5, H=320, I=160, E=12, K=3, seed=3),
    "replicas": dict(T=33, H=128, I=128, E=8, K=4, seed=4, extra=3),
    "skewed": dict(T=200, H=256, I=64, E=10, K=2, seed=5, skew=3.0),
    "many_rows": dict(T=700, H=128, I=96, E=4, K=2, seed=6),
    "large_tiles": dict(T=900, H=160, I=672, E=6, K=4, seed=17),
    "share": dict(T=64, H=192, I=64, E=32, K=8, seed=7, ep=2, extra=2),
    "wide_k": dict(T=9, H=64, I=32, E=64, K=32, seed=8),
    "one_expert": dict(T=40, H=1024, I=512, E=1, K=1, seed=9),
}


@pytest.mark.parametrize("name", LAYERS)
def test_layer_against_oracle(name):
    dev = device()
    spec = LAYERS[name]
    announce(f"mxfp4 layer {name} {spec}")
    T, K = spec["T"], spec["K"]
    L = _layer(**spec)
    ids, w = oracle.route(L["logits"], K, True)
    for rank in range(L["cfg"]["ep_size"]):
        want, tol = _reference(L, T, ids, w, rank)
        got = np64(_run(dev, L, T, rank, logits=L["logits"]))
        assert (np.abs(got - want) <= tol + 2.0 ** -8 * (np.abs(want) + tol)).all(), rank
    # routing given; f32 output; a shared output, accumulated into a given one
    shared = _rows(T, spec["H"], 5)
    base = torch.randn(T, spec["H"], generator=torch.Generator().manual_seed(6))
    out = base.to(dev)
    _run(dev, L, T, 0, topk_ids=torch.from_numpy(ids.astype(np.int32)), topk_w=torch.from_numpy(w.astype(np.float32)),
         shared_out=shared, out=out, cfg=dict(out_dtype=torch.float32, accumulate=True))
    want, tol = _reference(L, T, ids, w)
    want = want + np64(shared) + np64(base)
    assert (np.abs(np64(out) - want) <= tol + 8 * U * (np.abs(want) + np.abs(np64(base)) + np.abs(np64(shared)))).all()


def test_layer_shares_sum_to_the_whole():
    dev = device()
    announce("mxfp4 layer EP shares")
    spec = LAYERS["share"]
    L = _layer(**spec)
    W = _layer(**{**spec, "ep": 1, "extra": 0})
    whole = _run(dev, W, 64, logits=W["logits"], cfg=dict(out_dtype=torch.float32))
    acc = torch.zeros_like(whole)
    for r in range(2):
        _run(dev, L, 64, r, logits=L["logits"], out=acc, cfg=dict(out_dtype=torch.float32, accumulate=True))
    ids, w = oracle.route(W["logits"], spec["K"], True)
    _, tol = _reference(W, 64, ids, w)
    # the activations are the same bits, so only sums of f32 differ: far inside the allowance
    assert (np.abs(np64(acc) - np64(whole)) <= 0.05 * tol + 1e-6).all()


def test_layer_routing_on_input():
    dev = device()
    announce("mxfp4 layer routing on input")
    spec = LAYERS["few"]
    L = _layer(**spec)
    ids, w = oracle.route(L["logits"], 3, True)
    wt = torch.from_numpy(w.astype(np.float32))
    got = np64(_run(dev, L, 5, topk_ids=torch.from_numpy(ids.astype(np.int32)), topk_w=wt,
                    cfg=dict(routing_on_input=True)))
    want, tol = _reference(L, 5, ids, np64(wt), on_input=True)
    assert (np.abs(got - want) <= tol + 2.0 ** -8 * (np.abs(want) + tol)).all()


@pytest.mark.parametrize("T,I", [(1, 96), (5, 96), (60, 96), (300, 96), (900, 96), (950, 672)])
def test_layer_keeps_rows_apart(T, I):
    """A token of NaN and one of infinities change no other token's bits, whichever kernels run; and an
    expert whose slot the table does not give takes no part."""
    dev = device()
    announce(f"mxfp4 layer rows apart T={T} I={I}")
    H, E, K = 192, 8, 3
    L = _layer(T + 2, H, I, E, K, 31)
    a, b = T // 2, T + 1
    clean = _run(dev, L, T + 2, logits=L["logits"])
    x = L["x"].clone()
    L["x"][a] = float("nan")
    L["x"][b] = float("inf")
    got = _run(dev, L, T + 2, logits=L["logits"])
    rest = [t for t in range(T + 2) if t not in (a, b)]
    assert torch.equal(got[rest], clean[rest])
    assert torch.isnan(got[a]).all() and not torch.isfinite(got[b]).any()
    L["x"] = x
    bad = dict(L)
    bad["rs"] = L["rs"].clone()
    bad["rs"][2], bad["rs"][5] = 99, -7
    ids, w = oracle.route(L["logits"], K, True)
    w[(ids == 2) | (ids == 5)] = 0.0
    want, tol = _reference(L, T + 2, ids, w)
    got = np64(_run(dev, bad, T + 2, logits=L["logits"]))
    assert (np.abs(got - want) <= tol + 2.0 ** -8 * (np.abs(want) + tol) + 1e-38).all()


@pytest.mark.parametrize("T", [1, 2, 7, 200])
def test_layer_grouped_routing(T):
    dev = device()
    announce(f"mxfp4 layer grouped routing T={T}")
    L = _layer(T, 64, 32, 16, 3, 41)
    ids, w = oracle.route_grouped(L["logits"], 3, True, 4, 2)
    want, tol = _reference(L, T, ids, w)
    got = np64(_run(dev, L, T, logits=L["logits"], cfg=dict(num_expert_group=4, topk_group=2)))
    assert (np.abs(got - want) <= tol + 2.0 ** -8 * (np.abs(want) + tol) + 1e-38).all()


@pytest.mark.parametrize("E,K", [(1, 1), (6, 6), (8, 2), (60, 4), (64, 8), (64, 9), (96, 8), (128, 16), (130, 2),
                                 (256, 8), (200, 32), (300, 4)])
@pytest.mark.parametrize("renormalize", [True, False])
def test_few_tokens_in_every_router_form(E, K, renormalize):
    """One and two tokens, whose products route for themselves where lanes of a wave hold the experts: the bits
    of the same call on routed ids and weights, with logits that tie, one of two tokens with a NaN, a slot table that gives an
    expert no slot, and a share."""
    dev = device()
    announce(f"mxfp4 few tokens E={E} K={K} renormalize={renormalize}")
    for T in (1, 2):
        for ep in (1, 2):
            if E % ep:
                continue
            L = _layer(T, 64, 32, E, K, 51 + T, ep=ep, extra=1)
            L["logits"][:, E // 3:2 * E // 3] = 0.5
            if E > K and T == 2:
                L["logits"][0, E - 1] = float("nan")
            L["rs"] = L["rs"].clone()
            L["rs"][-1] = 10 ** 6
            ids, w = moe.route(L["logits"].to(dev), K, renormalize)
            for rank in range(ep):
                cfg = dict(out_dtype=torch.float32, renormalize=renormalize)
                got = _run(dev, L, T, rank, logits=L["logits"], cfg=cfg)
                want = _run(dev, L, T, rank, topk_ids=ids, topk_w=w, cfg=cfg)
                assert torch.equal(torch.nan_to_num(got, 7e9), torch.nan_to_num(want, 7e9)), (T, ep, rank)


def test_layer_is_its_stages():
    """forward against route, slot_map, permute, the two products and combine called one by one."""
    dev = device()
    announce("mxfp4 layer stages")
    for spec in (LAYERS["replicas"], LAYERS["one_token"], LAYERS["many_rows"]):
        T, K = spec["T"], spec["K"]
        L = _layer(**spec)
        S = L["cfg"]["S"]
        got = _run(dev, L, T, logits=L["logits"], cfg=dict(out_dtype=torch.float32))
        ids, w = moe.route(L["logits"].to(dev), K, True)
        slot, wm, mask = moe.slot_map(ids, w, spec["E"], rep_off=L["ro"].to(dev), rep_slots=L["rs"].to(dev))
        off, _, pr, xp = moe.permute(L["x"].to(dev), slot, mask, S)
        at = L["se"]
        a = moe.grouped_gemm_mxfp4(0, xp, off, L["gu"][at].to(dev), L["gs"][at].to(dev))
        y = moe.grouped_gemm_mxfp4(1, a, off, L["wd"][at].to(dev), L["ds"][at].to(dev), c_dtype=torch.float32)
        want = moe.combine(y, pr, wm, K)
        # the sums may be split differently: f32 steps, and activations that round the other way
        i, ww = oracle.route(L["logits"], K, True)
        _, tol = _reference(L, T, i, ww)
        assert (np.abs(np64(got) - np64(want)) <= tol).all()
        assert np.abs(np64(got) - np64(want)).mean() <= 0.02 * tol.mean()


def test_layer_empty_masked_and_workspace_reuse():
    dev = device()
    announce("mxfp4 layer empty and masked")
    L = _layer(**LAYERS["share"])
    # every pair of another rank: zeros, or the shared output alone
    ids = torch.full((64, 8), 31, dtype=torch.int32)
    w = torch.rand(64, 8)
    assert not _run(dev, L, 64, 0, topk_ids=ids, topk_w=w).any()
    sh = _rows(64, 192, 3)
    assert torch.equal(_run(dev, L, 64, 0, topk_ids=ids, topk_w=w, shared_out=sh).cpu(), sh)
    cfg = moe.ForwardConfig(T=0, T_max=64, **L["cfg"])
    assert moe.forward_workspace_size(cfg) > 0
    at = L["se"]
    a = [t.to(dev) for t in (L["gu"][at], L["wd"][at], L["gs"][at], L["ds"][at], L["ro"], L["rs"])]
    kw = dict(rep_off=a[4], rep_slots=a[5], w_gate_up_scale=a[2], w_down_scale=a[3])
    none = moe.forward(cfg, L["x"][:0].to(dev), a[0], a[1], logits=L["logits"][:0].to(dev), **kw)
    assert none.shape == (0, 192)
    # one workspace for calls of every size, whatever the last one left in it
    ws = torch.full((moe.forward_workspace_size(cfg),), 255, dtype=torch.uint8, device=dev)
    for T in (64, 1, 17, 2, 40):
        c = moe.ForwardConfig(T=T, T_max=64, **L["cfg"])
        got = moe.forward(c, L["x"][:T].to(dev), a[0], a[1], logits=L["logits"][:T].to(dev), ws=ws, **kw)
        fresh = moe.forward(moe.ForwardConfig(T=T, **L["cfg"]), L["x"][:T].to(dev), a[0], a[1],
                            logits=L["logits"][:T].to(dev), **kw)
        assert torch.equal(got, fresh), T


@pytest.mark.parametrize("T", [1, 6, 96, 600])
def test_layer_captured_in_a_graph_and_on_two_streams(T):
    """A decoding step, norm to layer, captured once and replayed on new inputs, eager work between;
    and two layers at once on two streams, each with its own workspace."""
    dev = device()
    announce(f"mxfp4 layer graph T={T}")
    H, I, E, K = 256, 128, 16, 4
    L = _layer(T, H, I, E, K, 21)
    cfg = moe.ForwardConfig(T=T, **L["cfg"])
    gu, wd, gs, ds, logits, x, res = (t.to(dev) for t in (L["gu"], L["wd"], L["gs"], L["ds"], L["logits"], L["x"],
                                                          _rows(T, H, 7)))
    gamma = torch.ones(H, dtype=torch.bfloat16, device=dev)

    def step():
        y, r, _ = moe.rms_norm(x, gamma, 1e-6, residual=res)
        return moe.forward(cfg, y, gu, wd, logits=logits, w_gate_up_scale=gs, w_down_scale=ds, shared_out=r)
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
        x.copy_(torch.randn(T, H, generator=g, device=dev))
        logits.copy_(torch.randn(T, E, generator=g, device=dev))
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        assert torch.equal(got, step())
    want = step()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        for s in streams:
            with torch.cuda.stream(s):
                outs.append(step())
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)


def test_layer_refusals():
    dev = device()
    L = _layer(**LAYERS["few"])
    cfg = moe.ForwardConfig(T=5, **L["cfg"])
    a = [t.to(dev) for t in (L["x"], L["gu"], L["wd"], L["gs"], L["ds"], L["logits"])]
    ok = dict(logits=a[5], w_gate_up_scale=a[3], w_down_scale=a[4])
    moe.forward(cfg, a[0], a[1], a[2], **ok)
    with pytest.raises(TypeError):
        moe.forward(cfg, a[0].float(), a[1], a[2], **ok)
    with pytest.raises(TypeError):
        moe.forward(cfg, a[0], a[1], a[2], **{**ok, "w_down_scale": None})
    with pytest.raises(TypeError):
        moe.forward(cfg, a[0], a[1], a[2], **{**ok, "w_down_scale": a[4].float()})
    with pytest.raises(ValueError):
        moe.forward(cfg, a[0], a[2], a[1], **ok)
    with pytest.raises(ValueError):
        moe.forward(cfg, a[0], a[1], a[2], **{**ok, "w_gate_up_scale": a[3][:, :, :1].contiguous()})


def test_layer_of_one_rank_of_very_many_pairs():
    """One of 1024 ranks, all 1024 slots its one expert's, 25 M pairs: the grid for the tiles that they could fill
    passes the 2^32 threads of one dimension. Half of them are here, so later tiles have rows."""
    dev = device()
    announce("mxfp4 layer 25 M pairs, one of 1024 ranks")
    if torch.cuda.mem_get_info()[0] < 100 * 2 ** 30:
        pytest.skip("needs 100 GiB of device memory")
    T, K, H, I, S = 24 * 1024 * 32, 32, 32, 1408, 1024
    gu, gs = _weights((1, 2 * I, H), 1, H)
    wd, ds = _weights((1, H, I), 2, I)
    x = _rows(T, H, 3)
    ids = torch.full((T, K), 5, dtype=torch.int32)
    ids[:, ::2] = 0
    w = torch.rand(T, K, generator=torch.Generator().manual_seed(4))
    cfg = moe.ForwardConfig(T=T, H=H, I=I, E_global=1024, K=K, renormalize=True, S=S, dtype=moe.MXFP4, ep_size=1024)
    slots = lambda t: t.to(dev).expand(S, -1, -1).contiguous()  # noqa: E731
    out = moe.forward(cfg, x.to(dev), slots(gu), slots(wd), topk_ids=ids.to(dev), topk_w=w.to(dev),
                      rep_off=torch.tensor([0, S], dtype=torch.int32, device=dev),
                      rep_slots=torch.arange(S, dtype=torch.int32, device=dev),
                      w_gate_up_scale=slots(gs), w_down_scale=slots(ds))
    some = torch.arange(0, T, 8191)
    some[-1] = T - 1
    n = some.numel()
    L = dict(gu=gu, gs=gs, wd=wd, ds=ds, x=x[some], El=1, cfg=dict(H=H, I=I))
    # the same row K / 2 times: once, with the weights' sum (K / 2 - 1 more additions in f32)
    want, tol = _reference(L, n, np.zeros((n, 1), int), np64(w[some])[:, ::2].sum(1, keepdims=True))
    got = np64(out[some.to(dev)])
    assert (np.abs(got - want) <= tol * (1 + K * U) + 2.0 ** -8 * (np.abs(want) + tol) + 1e-38).all()
    del out
    torch.cuda.empty_cache()


# ------------------------------------------------------------------ pair by pair
def _taken_pair_by_pair(dev, L, T, **kw):
    """Whether a call goes pair by pair, by what it writes into its workspace: routing and activations, but no
    expert output of each pair ([T * K, H] f32)."""
    P, H, I = T * L["cfg"]["K"], L["cfg"]["H"], L["cfg"]["I"]
    assert 7 * H // 2 > 17 + 2 * I
    cfg = moe.ForwardConfig(T=T, **L["cfg"])
    ws = torch.full((moe.forward_workspace_size(cfg),), 0xA5, dtype=torch.uint8, device=dev)
    out = _run(dev, L, T, ws=ws, **kw)
    return out, int((ws != 0xA5).sum()) <= P * (17 + 2 * I)


# H in each form of the gate/up product (up to 2048, 4096, more), over whole and broken steps of 128, 256 and 512
@pytest.mark.parametrize("H", [608, 1184, 2048, 2080, 2560, 3968, 4096, 4128, 6176])
@pytest.mark.parametrize("T,K,I", [(1, 3, 608), (2, 2, 32), (1, 1, 928), (2, 4, 352)])
def test_pairs_of_wide_rows(H, T, K, I):
    dev = device()
    announce(f"mxfp4 pairs T={T} K={K} H={H} I={I}")
    L = _layer(T, H, I, K + 1, K, H + I)
    got, pairs = _taken_pair_by_pair(dev, L, T, logits=L["logits"])
    assert pairs
    ids, w = oracle.route(L["logits"], K, True)
    want, tol = _reference(L, T, ids, w)
    assert (np.abs(np64(got) - want) <= tol + 2.0 ** -8 * (np.abs(want) + tol)).all()


# (T, K, H, I, pair by pair): at and just past 64 pairs, 16 M weights of one matrix over all pairs and
# 768 blocks of 32 or 16 columns
BOUNDS = [(16, 4, 256, 64, True), (13, 5, 256, 64, False), (64, 1, 320, 32, True), (65, 1, 320, 32, False),
          (16, 4, 1024, 256, True), (16, 4, 1024, 288, False), (16, 4, 672, 384, True), (16, 4, 608, 416, False),
          (5, 4, 2080, 384, True), (5, 4, 2080, 416, False), (4, 5, 4096, 192, True), (5, 4, 4128, 192, True),
          (3, 2, 5216, 512, True), (3, 2, 5216, 544, False), (24, 2, 2080, 160, True), (10, 6, 2048, 128, True)]


@pytest.mark.parametrize("T,K,H,I,pairs", BOUNDS)
def test_pairs_at_their_bounds(T, K, H, I, pairs):
    """Both sides of each bound, routed here and with given ids, with replicated slots, against the oracle."""
    dev = device()
    announce(f"mxfp4 pair bounds T={T} K={K} H={H} I={I}")
    L = _layer(T, H, I, 8, K, T + K + H + I, extra=2)
    ids, w = oracle.route(L["logits"], K, True)
    want, tol = _reference(L, T, ids, w)
    for kw in (dict(logits=L["logits"]),
               dict(topk_ids=torch.from_numpy(ids.astype(np.int32)), topk_w=torch.from_numpy(w.astype(np.float32)))):
        got, taken = _taken_pair_by_pair(dev, L, T, **kw)
        assert taken == pairs
        assert (np.abs(np64(got) - want) <= tol + 2.0 ** -8 * (np.abs(want) + tol)).all()


# ------------------------------------------------------------------ stage events
@pytest.mark.parametrize("T", [1, 2, 16])
@pytest.mark.parametrize("given", [False, True])
def test_stage_events_follow_their_stages(T, given):
    """An event is recorded behind the launch that ends its stage: the weights that a product has to read, at
    25 TB/s (three times what the memory gives; they pass every L2), are a time that has to lie between the
    events around it."""
    dev = device()
    announce(f"mxfp4 events T={T} given={given}")
    H, I, K, E = 8192, 16384, 4, 8
    g = torch.Generator(device=dev).manual_seed(T)
    byte = lambda *s: torch.randint(0, 256, s, generator=g, device=dev, dtype=torch.uint8)  # noqa: E731
    sc = lambda *s: torch.randint(118, 121, s, generator=g, device=dev, dtype=torch.uint8)  # noqa: E731
    w = (byte(E, 2 * I, H // 2), byte(E, H, I // 2))
    kw = dict(w_gate_up_scale=sc(E, 2 * I, H // 32), w_down_scale=sc(E, H, I // 32))
    x = torch.randn(T, H, generator=g, device=dev).bfloat16()
    logits = torch.randn(T, E, generator=g, device=dev)
    if given:
        kw["topk_ids"], kw["topk_w"] = moe.route(logits, K, True)
    else:
        kw["logits"] = logits
    cfg = moe.ForwardConfig(T=T, H=H, I=I, E_global=E, K=K, renormalize=True, S=E, dtype=moe.MXFP4)
    ev = [torch.cuda.Event(enable_timing=True) for _ in range(moe.NUM_EVENTS)]
    for e in ev:
        e.record()
    for _ in range(3):
        moe.forward(cfg, x, *w, events=[e.cuda_event for e in ev], **kw)
    torch.cuda.synchronize()
    us = [1e3 * a.elapsed_time(b) for a, b in zip(ev, ev[1:])]
    assert all(t >= 0 for t in us)
    down = K * H * I * 17 / 32 / 25e6       # at least K slots of one matrix: 11 us
    # routing and permutation stand before GATE_UP, in the gate/up launch or before it
    assert sum(us[:3]) >= 2 * down and us[3] + us[4] >= down and us[3] >= down, us
    if T <= 2 and not given:                # routed by the gate/up product: those stages end with it
        assert us[0] >= 2 * down, us
