"""Every entry point that launches work is called in one place, which makes its tensors' device the current one,
passes that device's stream and refuses tensors of two devices. Seen without a device: the calls get tensors
of the meta device and that place is replaced by one that notes what it is given.
"""
import pytest
import torch

import moe_expert_dispatch_amd as moe

B, F, I32, U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8


def _t(*shape, dt=B):
    return torch.empty(*shape, dtype=dt, device="meta")


@pytest.fixture
def seen(monkeypatch):
    calls = []
    sizes = type("Sizes", (), {"__getattr__": lambda self, name: (lambda *a: 16)})()  # workspace sizes alone
    monkeypatch.setattr(moe, "_dev", lambda t, name, dtype=None, shape=None: t)
    monkeypatch.setattr(moe, "_lib", sizes)
    monkeypatch.setattr(moe, "_launch", lambda what, like, others, *args: calls.append((what, like, others, args)))
    return calls


def _stage_calls():
    x, ids, w = _t(6, 16), _t(6, 2, dt=I32), _t(6, 2, dt=F)
    slot, mask, ws = _t(6, 2, dt=I32), _t(6, 2, dt=U8), _t(64, dt=U8)
    off, pr, y = _t(5, dt=I32), _t(12, dt=I32), _t(12, 16)
    gu, wd, codes = _t(4, 16, 16), _t(4, 16, 8), _t(12, 16, dt=U8)
    ro, rs, sc, xs = _t(4, dt=I32), _t(4, dt=I32), _t(4, dt=F), _t(6, 16)
    out = (_t(5, dt=I32), _t(12, dt=I32), _t(12, dt=I32), _t(12, 16))
    return {
        "moe_route": (lambda: moe.route(w, 2, True, ids, w), (w, ids)),
        "moe_route_grouped": (lambda: moe.route(w, 2, True, ids, w, 2, 1), (w, ids)),
        "moe_slot_map": (lambda: moe.slot_map(ids, w, 4, rep_off=ro, rep_slots=rs), (ids, w, ro, rs)),
        "moe_permute": (lambda: moe.permute(x, slot, mask, 4, ws=ws), (x, slot, mask, ws)),
        "moe_permute_scaled": (lambda: moe.permute(x, slot, mask, 4, ws=ws, pair_w=w), (x, slot, mask, ws, w)),
        "moe_permute_noalloc": (lambda: moe.permute_noalloc(x, slot, mask, 4, out=out), (x, slot, mask, *out)),
        "moe_grouped_gemm": (lambda: moe.grouped_gemm(moe.DOWN, _t(12, 8), off, wd, y), (off, wd, y)),
        "moe_quantize_fp8": (lambda: moe.quantize_fp8(x, 1.0, codes), (x, codes)),
        "moe_grouped_gemm_fp8": (lambda: moe.grouped_gemm_fp8(moe.GATE_UP_SWIGLU, codes, 1.0, off, gu, sc), (codes, off, gu, sc)),
        "moe_combine": (lambda: moe.combine(y, pr, w, 2, out=x), (y, pr, w, x)),
        "moe_combine_shared": (lambda: moe.combine(y, pr, w, 2, out=x, shared=xs), (y, pr, w, x, xs)),
        "moe_a2a_dispatch": (lambda: moe.a2a_dispatch(x, ids, w, 4, 2, ws=ws), (x, ids, w, ws)),
        "moe_a2a_combine": (lambda: moe.a2a_combine(y, ids), (y, ids)),
    }


@pytest.mark.parametrize("what", list(_stage_calls()))
def test_stages(seen, what):
    call, tensors = _stage_calls()[what]
    call()
    (name, like, others, args), = seen
    assert name == what and len(args) == len(moe._SIGS[what][1]) - 1   # the stream is added behind them
    given = [like, *others]
    for t in tensors:
        assert any(t is g for g in given), "a tensor whose device is not looked at"
