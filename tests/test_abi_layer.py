"""Host validation of the norm, the router's loss and gradient, and the MXFP4
entry points: every call here fails its checks, has no work, or asks a
workspace size, so nothing reaches a device.
"""
import ctypes
import os
import subprocess
import sys

import pytest
import torch

import moe_expert_dispatch_amd as moe

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3
fake = ctypes.c_void_p(256)
odd = ctypes.c_void_p(264)


@pytest.fixture(scope="module")
def so():
    return moe.lib()


def test_rms_norm_validation(so):
    def call(x=fake, res=fake, gamma=fake, dt=1, T=4, H=64, eps=1e-6, ro=fake, y=fake, q=fake,
             scale=0.5):
        return so.moe_rms_norm(x, res, gamma, dt, T, H, eps, ro, y, q, scale, None)
    assert call(T=-1) == INVALID
    assert call(H=0) == INVALID
    for eps in (-1e-6, float("nan"), float("inf")):
        assert call(eps=eps) == INVALID
    assert call(dt=2) == UNSUPPORTED and call(dt=3) == UNSUPPORTED
    assert call(H=60) == UNSUPPORTED and call(H=32776) == UNSUPPORTED
    assert call(x=None) == INVALID and call(gamma=None) == INVALID
    assert call(ro=None, y=None, q=None) == INVALID
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        assert call(scale=scale) == INVALID
    for k in ("x", "res", "gamma", "ro", "y", "q"):
        assert call(**{k: odd}) == INVALID
    assert call(T=0, x=None, gamma=None, scale=0.0) == 0


def test_scales_need_a_finite_reciprocal(so):
    """Codes are of v * (1 / scale): a scale below 2^-128 has no reciprocal in f32 (0 would get the code of NaN)."""
    other = ctypes.c_void_p(1 << 20)
    for s in (1e-39, 2.0 ** -128, 1e-45):
        assert so.moe_rms_norm(fake, None, other, 1, 4, 64, 1e-6, None, None, fake, s, None) == INVALID
        assert so.moe_quantize_fp8(fake, 1, 4, s, fake, None) == INVALID
        cfg = _cfg(H=256, I=256, dtype=moe.FP8, a2_scale=s)
        assert so.moe_forward_workspace_size(ctypes.byref(cfg.c_struct())) == 0
    for s in (2.0 ** -127, 2.0 ** -126, 3.0e38):
        cfg = _cfg(H=256, I=256, dtype=moe.FP8, a2_scale=s)
        assert so.moe_forward_workspace_size(ctypes.byref(cfg.c_struct())) > 0


def test_rms_norm_refuses_one_place_for_two_outputs(so):
    """residual_out may be x and y may be x, but not both at once."""
    other = ctypes.c_void_p(1 << 20)

    def call(ro, y):
        return so.moe_rms_norm(fake, other, other, 1, 4, 64, 1e-6, ro, y, None, 0.0, None)
    assert call(fake, fake) == INVALID and call(other, other) == INVALID


def test_balance_loss_validation(so):
    ws = so.moe_balance_loss_workspace_size
    assert ws(0, 8, 2) > 0 and ws(1 << 20, 1024, 32) > 0
    assert ws(-1, 8, 2) == 0 and ws(4, 8, 9) == 0 and ws(4, 1025, 2) == 0
    sizes = [ws(t, 60, 4) for t in range(0, 20000, 331)]
    assert all(a <= b for a, b in zip(sizes, sizes[1:]))

    def call(l=fake, i=fake, m=fake, T=4, E=8, K=2, c=fake, p=fake, loss=fake, w=fake,
             n=ctypes.c_size_t(1 << 20)):
        return so.moe_balance_loss(l, i, m, T, E, K, 1.0, c, p, loss, w, n, None)
    assert call(T=-1) == INVALID and call(K=0) == INVALID and call(K=9) == INVALID
    assert call(E=1025) == UNSUPPORTED and call(E=64, K=33) == UNSUPPORTED
    for k in ("l", "i", "c", "p", "loss"):
        assert call(**{k: None}) == INVALID
    assert call(w=None) == WORKSPACE
    assert call(n=ctypes.c_size_t(ws(4, 8, 2) - 1)) == WORKSPACE
    assert call(w=odd) == INVALID


def test_route_backward_validation(so):
    def call(l=fake, i=fake, dw=fake, c=fake, T=4, E=8, K=2, d=fake):
        return so.moe_route_backward(l, i, dw, None, c, None, T, E, K, 1, 1.0, d, None)
    assert call(T=-1) == INVALID and call(K=9) == INVALID
    assert call(E=2048) == UNSUPPORTED
    assert call(dw=None, c=None) == INVALID
    assert call(l=None) == INVALID and call(d=None) == INVALID and call(i=None) == INVALID
    assert call(T=0, l=None, d=None) == 0


def test_mxfp4_weight_validation(so):
    for f in (lambda w, dt, n, c, s: so.moe_quantize_mxfp4(w, dt, n, c, s, None),
              lambda w, dt, n, c, s: so.moe_dequantize_mxfp4(c, s, n, w, dt, None)):
        assert f(fake, 1, -32, fake, fake) == INVALID
        assert f(fake, 1, 48, fake, fake) == UNSUPPORTED
        assert f(fake, 2, 64, fake, fake) == UNSUPPORTED
        assert f(fake, 1, 1 << 40, fake, fake) == UNSUPPORTED
        assert f(None, 1, 64, fake, fake) == INVALID
        assert f(odd, 0, 64, fake, fake) == INVALID
        assert f(fake, 0, 64, odd, fake) == INVALID
        assert f(fake, 0, 64, fake, odd) == INVALID
        assert f(None, 0, 0, None, None) == 0


def test_grouped_gemm_mxfp4_validation(so):
    def call(op=0, S=4, rows=16, H=64, I=64, a=fake, w=fake, ws=fake, c=fake, cdt=1, off=fake):
        return so.moe_grouped_gemm_mxfp4(op, a, off, S, rows, w, ws, H, I, c, cdt, None)
    assert call(op=5) == INVALID and call(S=0) == INVALID and call(rows=-1) == INVALID
    assert call(H=72) == UNSUPPORTED and call(I=40) == UNSUPPORTED
    assert call(S=1025) == UNSUPPORTED
    assert call(cdt=0) == UNSUPPORTED               # gate/up writes bf16
    assert call(op=1, cdt=2) == UNSUPPORTED
    assert call(off=None) == INVALID
    for k in ("a", "w", "ws", "c"):
        assert call(**{k: None}) == INVALID and call(**{k: odd}) == INVALID
    assert call(rows=0) == 0 and call(op=1, rows=0, cdt=0) == 0
    assert call(rows=0, H=32768, I=32768) == UNSUPPORTED  # the weight-panel limit, one byte a weight


def test_grouped_gemm_mxfp4_refuses_rows_whose_tiles_pass_31_bits(so):
    """Tiles step past a slot's last row by up to 160 rows, in 32-bit indices. The check behind this one (no scales)
    refuses the rest without a launch."""
    def call(rows):
        return so.moe_grouped_gemm_mxfp4(1, fake, fake, 4, rows, fake, None, 64, 64, fake, 1, None)
    for rows in (2 ** 31 - 1, 2 ** 31 - 1024):
        assert call(rows) == UNSUPPORTED
    assert call(2 ** 31 - 1025) == INVALID


def _cfg(**kw):
    base = dict(T=16, H=64, I=64, E_global=8, K=2, renormalize=True, S=8, dtype=moe.MXFP4)
    base.update(kw)
    return moe.ForwardConfig(**base)


def test_forward_config_validation(so):
    size = lambda c: so.moe_forward_workspace_size(ctypes.byref(c.c_struct()))  # noqa: E731
    ok = _cfg()
    assert ok.out_dtype == torch.bfloat16
    n = size(ok)
    assert n >= 32 * 64 * 4 + 32 * 64 * 2  # f32 expert outputs, bf16 activations
    for bad in (_cfg(H=72), _cfg(I=72), _cfg(x_codes=True), _cfg(dtype=torch.bfloat16, x_codes=True),
                _cfg(out_dtype=moe.MXFP4)):
        assert size(bad) == 0
    args = moe._ForwardArgs()
    for name in ("x", "logits", "w_gate_up", "w_down", "out", "w_gate_up_e8m0", "w_down_e8m0"):
        setattr(args, name, 256)
    call = lambda: so.moe_forward(ctypes.byref(ok.c_struct()), ctypes.byref(args),  # noqa: E731
                                  ctypes.c_void_p(256), n, None)
    for name in ("w_gate_up_e8m0", "w_down_e8m0"):
        for v in (None, 264):
            setattr(args, name, v)
            assert call() == INVALID
        setattr(args, name, 256)
    # FP8 with codes for x needs no room for its own
    fp8 = dict(H=256, I=256, dtype=moe.FP8)
    assert size(_cfg(**fp8, x_codes=True)) == size(_cfg(**fp8)) - 16 * 256


def test_python_layer_refuses(so):
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        moe.rms_norm(x, x[0])
    with pytest.raises(ValueError):
        moe.quantize_mxfp4(x)
    with pytest.raises(TypeError):
        moe.quantize_mxfp4([1.0])
    with pytest.raises(ValueError):
        moe.balance_loss(x.float(), torch.zeros(4, 2, dtype=torch.int32), 1.0)
    with pytest.raises(ValueError):
        moe.route_backward(x.float(), torch.zeros(4, 2, dtype=torch.int32), None, True)


def test_balance_loss_workspace_at_the_most_tokens(so):
    """T * K < 2^31: the largest T takes the blocks, and with them the workspace, of every large T."""
    ws = so.moe_balance_loss_workspace_size
    for E, K in ((1, 1), (8, 1), (64, 1)):
        assert ws(2 ** 31 - 1, E, K) == ws(2 ** 30, E, K) > ws(64, E, K)


@pytest.mark.parametrize("S", [1, 80, 1024])
def test_permute_refuses_pairs_whose_chunks_pass_31_bits(so, S):
    """A chunk's end, first pair + chunk, is a 32-bit index: the last chunk of 2^31 - 1 pairs ends behind it."""
    ws = so.moe_permute_workspace_size
    small = ws(1 << 30, 1, S)
    assert small >= 4 * S

    def call(T, K=1, n=0):
        return so.moe_permute(None, 1, T, 64, K, fake, fake, S, fake, fake, fake, None, fake, ctypes.c_size_t(n), None)
    for T, K in ((2 ** 31 - 1, 1), (2 ** 31 - 600, 1), ((2 ** 31 - 1) // 7, 7), (2 ** 26 - 1, 32)):
        assert ws(T, K, S) == 0 and call(T, K, 1 << 40) == UNSUPPORTED
        assert so.moe_permute_noalloc(None, 1, T, 64, K, fake, fake, S, fake, fake, fake, None, None) != 0
        cfg = moe.ForwardConfig(T=T, H=32, I=32, E_global=max(K, 1), K=K, renormalize=True, S=max(S, K), dtype=moe.MXFP4)
        assert so.moe_forward_workspace_size(ctypes.byref(cfg.c_struct())) == 0
    # the most that is taken: chunks of T / n tokens, n = 65536 / S, and the steps past the end of one
    n = 65536 // S
    most = max(T for T in range(2 ** 31 - 2 ** 26, 2 ** 31, 1 << 12) if T + -(-T // n) + 1024 < 2 ** 31)
    assert ws(most, 1, S) == small and call(most) == WORKSPACE


def test_a2a_dispatch_refuses_more_tokens_than_its_grid_holds(so):
    """A block of 256 threads a token, and up to 256 more: 2^32 threads from 2^24 - 256 tokens on."""
    most = (1 << 24) - 257
    ws = so.moe_a2a_dispatch_workspace_size
    assert ws(most, 1, most) > 0 and ws(most + 1, 1, most + 1) == 0

    def call(T, n):
        return so.moe_a2a_dispatch(fake, 1, T, 64, 1, fake, fake, 8, 1, T, fake, fake, fake, fake, fake, fake, fake,
                                   ctypes.c_size_t(n), None)
    assert call(most, 0) == WORKSPACE
    assert call(most + 1, 0) == UNSUPPORTED and call(1 << 24, 1 << 40) == UNSUPPORTED


def test_package_needs_no_torch_type_of_four_bits():
    """A torch without float4_e2m1fn_x2: the package imports, and MXFP4 still names its layers."""
    code = """
import torch
del torch.float4_e2m1fn_x2
import ctypes, moe_expert_dispatch_amd as moe
size = lambda dt: moe.lib().moe_forward_workspace_size(ctypes.byref(moe.ForwardConfig(
    T=16, H=64, I=64, E_global=8, K=2, renormalize=True, S=8, dtype=dt).c_struct()))
assert moe.ForwardConfig(16, 64, 64, 8, 2, True, 8, moe.MXFP4).out_dtype == torch.bfloat16
print(size(moe.MXFP4), size(torch.bfloat16), size(torch.float32))
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    run = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=100)
    assert run.returncode == 0, run.stderr
    sizes = [int(v) for v in run.stdout.split()]
    here = [moe.lib().moe_forward_workspace_size(ctypes.byref(_cfg(dtype=dt).c_struct()))
            for dt in (moe.MXFP4, torch.bfloat16, torch.float32)]
    assert sizes == here and all(sizes)
