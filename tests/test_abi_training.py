"""Host validation of the layer's training pass: every call here fails its checks, has no work, or asks a
workspace size, so nothing reaches a device.
"""
import ctypes

import pytest
import torch

import moe_expert_dispatch_amd as moe

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3
a, b, c, d, e, f, g = (ctypes.c_void_p(256 * (i + 1)) for i in range(7))
odd = ctypes.c_void_p(264)
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def so():
    return moe.lib()


def test_layer_norm(so):
    def call(x=a, res=b, gamma=c, beta=d, dt=1, T=4, H=64, eps=1e-6, ro=e, y=f, q=g, scale=0.5):
        return so.moe_layer_norm(x, res, gamma, beta, dt, T, H, eps, ro, y, q, scale, None)
    assert call(T=-1) == INVALID and call(H=0) == INVALID
    for eps in (-1e-6, NAN, INF):
        assert call(eps=eps) == INVALID
    assert call(dt=2) == UNSUPPORTED and call(H=60) == UNSUPPORTED and call(H=32776) == UNSUPPORTED
    assert call(x=None) == INVALID and call(gamma=None) == INVALID
    assert call(ro=None, y=None, q=None) == INVALID
    assert call(ro=f) == INVALID  # two outputs in one place
    for scale in (0.0, -1.0, NAN, INF, 2.0 ** -128):
        assert call(scale=scale) == INVALID
    for k in ("x", "res", "gamma", "beta", "ro", "y", "q"):
        assert call(**{k: odd}) == INVALID
    assert call(T=0, x=None, gamma=None, scale=0.0) == 0


@pytest.mark.parametrize("layer", [False, True])
def test_norm_backward(so, layer):
    need = moe.norm_backward_workspace_size(4, 64)

    def call(dy=a, x=b, gamma=c, dres=d, dt=1, T=400, H=4096, eps=1e-6, dx=e, dgamma=f, dbeta=g, ws=a,
             size=1 << 30):
        last = (dgamma, dbeta) if layer else (dgamma,)
        fn = so.moe_layer_norm_backward if layer else so.moe_rms_norm_backward
        return fn(dy, x, gamma, dres, dt, T, H, eps, dx, *last, ws, size, None)
    assert call(T=-1) == INVALID and call(H=0) == INVALID
    for eps in (-1e-6, NAN, INF):
        assert call(eps=eps) == INVALID
    assert call(dt=3) == UNSUPPORTED and call(H=60) == UNSUPPORTED and call(H=32776) == UNSUPPORTED
    for k in ("dy", "x", "gamma"):
        assert call(**{k: None}) == INVALID
    for k in ("dy", "x", "gamma", "dres", "dx", "dgamma", "ws"):
        assert call(**{k: odd}) == INVALID, k
    assert call(dx=None, dgamma=None, dbeta=None) == INVALID
    assert call(ws=None) == WORKSPACE
    size = moe.norm_backward_workspace_size(400, 4096)
    assert size % (2 * 4096 * 4) == 0 and 0 < size <= 400 * 2 * 4096 * 4 and call(size=size - 1) == WORKSPACE
    if layer:
        assert call(dbeta=f) == INVALID
    assert call(T=0, dgamma=None, dbeta=None, dy=None, x=None, gamma=None, ws=None, size=0) == 0
    assert need == 0  # few rows: one launch, no partial sums
    for T, H in ((-1, 64), (4, 0), (4, 60), (4, 32776)):
        assert moe.norm_backward_workspace_size(T, H) == 0


def test_norm_backward_workspace_is_bounded():
    for H in (8, 128, 512, 520, 4096, 8192, 16384, 32768):
        sizes = [moe.norm_backward_workspace_size(T, H) for T in (0, 1, 1000, 10 ** 6, 2 ** 31 - 1)]
        assert sizes == sorted(sizes) and sizes[-1] <= 1024 * 2 * H * 4


def test_combine_backward(so):
    def call(dout=a, ddt=1, y=b, ydt=1, pr=c, w=d, T=4, K=2, H=64, dy=e, dw=f):
        return so.moe_combine_backward(dout, ddt, y, ydt, pr, w, T, K, H, dy, dw, None)
    assert call(T=-1) == INVALID and call(K=0) == INVALID and call(H=0) == INVALID
    assert call(ddt=2) == UNSUPPORTED and call(ydt=3) == UNSUPPORTED
    assert call(K=33) == UNSUPPORTED and call(H=60) == UNSUPPORTED and call(H=1 << 24) == UNSUPPORTED
    assert call(T=1 << 30, K=2) == UNSUPPORTED
    for k in ("dout", "pr", "y"):
        assert call(**{k: None}) == INVALID
    assert call(dy=None, dw=None) == INVALID
    for k in ("dout", "y", "dy"):
        assert call(**{k: odd}) == INVALID
    assert call(dy=b) == INVALID and call(dy=a) == INVALID
    assert call(T=0, dout=None, pr=None, y=None, dy=None, dw=None) == 0


def test_permute_backward(so):
    def call(dxp=a, dt=1, pr=b, w=c, x=d, T=4, K=2, H=64, dx=e, xdt=0, acc=0, dw=f):
        return so.moe_permute_backward(dxp, dt, pr, w, x, T, K, H, dx, xdt, acc, dw, None)
    assert call(T=-1) == INVALID and call(K=0) == INVALID and call(H=0) == INVALID
    assert call(dt=2) == UNSUPPORTED and call(xdt=3) == UNSUPPORTED
    assert call(K=33) == UNSUPPORTED and call(H=60) == UNSUPPORTED and call(H=1 << 24) == UNSUPPORTED
    for k in ("dxp", "pr", "dx"):
        assert call(**{k: None}) == INVALID
    assert call(w=None) == INVALID and call(x=None) == INVALID  # dpair_w needs both
    for k in ("dxp", "x", "dx"):
        assert call(**{k: odd}) == INVALID
    assert call(dx=a) == INVALID and call(dx=d) == INVALID
    assert call(T=0, dxp=None, pr=None, dx=None) == 0


def test_swiglu(so):
    def call(h=a, dt=1, off=b, S=4, rows=8, I=64, act=c):
        return so.moe_swiglu(h, dt, off, S, rows, I, act, None)
    assert call(S=0) == INVALID and call(rows=-1) == INVALID and call(I=0) == INVALID
    assert call(dt=2) == UNSUPPORTED and call(S=1025) == UNSUPPORTED and call(I=60) == UNSUPPORTED
    assert call(I=1 << 20) == UNSUPPORTED and call(rows=2 ** 31 - 1024) == UNSUPPORTED
    for k in ("h", "off", "act"):
        assert call(**{k: None}) == INVALID
    for k in ("h", "act"):
        assert call(**{k: odd}) == INVALID
    assert call(act=a) == INVALID
    assert call(rows=0, h=None, act=None) == 0


def test_grouped_gemm_backward(so):
    def call(op=1, dt=1, dc=a, off=b, S=4, rows=8, w=c, H=64, I=32, h=d, out=e):
        return so.moe_grouped_gemm_backward(op, dt, dc, off, S, rows, w, H, I, h, out, None)
    assert call(op=2) == INVALID and call(op=0) == INVALID  # h belongs to the down product
    assert call(S=0) == INVALID and call(rows=-1) == INVALID and call(H=0) == INVALID and call(I=0) == INVALID
    assert call(dt=2) == UNSUPPORTED and call(S=1025) == UNSUPPORTED
    assert call(H=60) == UNSUPPORTED and call(I=60) == UNSUPPORTED
    assert call(rows=2 ** 31 - 1024) == UNSUPPORTED
    assert call(H=1 << 20, I=8) == UNSUPPORTED and call(op=0, h=None, I=1 << 19, H=8) == UNSUPPORTED
    assert call(H=32768, I=32768) == UNSUPPORTED            # a slot's panel of 2^31 bytes
    assert call(dt=0, H=16384, I=32768) == UNSUPPORTED
    assert call(rows=2 ** 31 - 2048, H=8, I=524288) == UNSUPPORTED   # tiles past 31 bits
    for k in ("dc", "off", "w", "out"):
        assert call(**{k: None}) == INVALID
    for k in ("dc", "w", "h", "out"):
        assert call(**{k: odd}) == INVALID
        if k != "out":
            assert call(out={"dc": a, "w": c, "h": d}[k]) == INVALID
    assert call(rows=0, dc=None, w=None, out=None) == 0


def test_weight_grad(so):
    def call(dt=1, dc=a, x=b, off=c, S=4, rows=8, N=64, Kd=32, dw=d, ddt=0, acc=0, ws=e, size=1 << 40):
        return so.moe_grouped_gemm_weight_grad(dt, dc, x, off, S, rows, N, Kd, dw, ddt, acc, ws, size, None)
    assert call(S=0) == INVALID and call(rows=-1) == INVALID and call(N=0) == INVALID and call(Kd=0) == INVALID
    assert call(dt=2) == UNSUPPORTED and call(ddt=2) == UNSUPPORTED and call(S=1025) == UNSUPPORTED
    assert call(N=60) == UNSUPPORTED and call(Kd=60) == UNSUPPORTED and call(N=1 << 20) == UNSUPPORTED
    assert call(Kd=1 << 20) == UNSUPPORTED and call(rows=2 ** 31 - 1024) == UNSUPPORTED
    assert call(S=1024, N=(1 << 20) - 8, Kd=(1 << 20) - 8) == UNSUPPORTED
    for k in ("dc", "x", "off", "dw"):
        assert call(**{k: None}) == INVALID
    for k in ("dc", "x", "dw"):
        assert call(**{k: odd}) == INVALID
    assert call(dw=a) == INVALID and call(dw=b) == INVALID
    need = moe.grouped_gemm_weight_grad_workspace_size(torch.bfloat16, 2, 1 << 17, 256, 128)
    assert need > 0 and need % (2 * 256 * 128 * 4) == 0
    assert call(S=2, rows=1 << 17, N=256, Kd=128, size=need - 1) == WORKSPACE
    assert call(S=2, rows=1 << 17, N=256, Kd=128, ws=None) == WORKSPACE
    assert call(S=2, rows=1 << 17, N=256, Kd=128, ws=odd) == INVALID
    assert moe.grouped_gemm_weight_grad_workspace_size(torch.bfloat16, 64, 1 << 17, 2048, 4096) == 0
    assert moe.grouped_gemm_weight_grad_workspace_size(torch.bfloat16, 2, 0, 256, 128) == 0


def test_bindings_refuse_host_tensors():
    x = torch.zeros(4, 64)
    pr = torch.zeros(8, dtype=torch.int32)
    for call in (lambda: moe.layer_norm(x, x[0]), lambda: moe.rms_norm_backward(x, x, x[0]),
                 lambda: moe.layer_norm_backward(x, x, x[0]), lambda: moe.combine_backward(x, x, pr, None, 2),
                 lambda: moe.permute_backward(x, pr, 2), lambda: moe.swiglu(x, pr),
                 lambda: moe.grouped_gemm_backward(moe.DOWN, x, pr, x[None]),
                 lambda: moe.grouped_gemm_weight_grad(x, x, pr)):
        with pytest.raises(ValueError, match="device"):
            call()
