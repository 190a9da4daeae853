"""Token counts whose launches pass the 2^32 threads of one grid dimension, for
the stages of the layer. The inputs repeat after a short period, and so have
the outputs to, which a small call gives.
"""
import pytest
import torch

import moe_expert_dispatch_amd as moe
from gpu_common import announce, device

pytestmark = pytest.mark.gpu

PERIOD = 1021


def _need(gib):
    if torch.cuda.mem_get_info()[0] < gib * 2 ** 30:
        pytest.skip(f"needs {gib} GiB of device memory")


def _repeat(part, n):
    """part [p, ...] again and again, to n rows."""
    whole, p = n // part.shape[0], part.shape[0]
    out = part.new_empty(n, *part.shape[1:])
    out[:whole * p].view(whole, *part.shape).copy_(part.expand(whole, *part.shape))
    out[whole * p:] = part[:n - whole * p]
    return out


def _repeats(got, part):
    whole, p = got.shape[0] // part.shape[0], part.shape[0]
    lines = got[:whole * p].view(whole, *part.shape)
    step = max(1, (1 << 31) // part.numel())
    return (all(bool((lines[i:i + step] == part).all()) for i in range(0, whole, step)) and
            torch.equal(got[whole * p:], part[:got.shape[0] - whole * p]))


def _free():
    torch.cuda.empty_cache()


# lane groups of 8 with 2^32 threads at 2^29 tokens, a wave a token at 2^26 (group-limited)
@pytest.mark.parametrize("T,E,groups", [(2 ** 29 + 7, 2, 0), (2 ** 26 + 7, 8, 4)])
def test_route(T, E, groups):
    dev = device()
    _need(24)
    announce(f"route T={T} E={E} groups={groups}")
    part = torch.randn(PERIOD, E, generator=torch.Generator().manual_seed(1)).to(dev)
    kw = dict(num_groups=groups, topk_groups=2) if groups else {}
    ids, w = moe.route(_repeat(part, T), 1, False, **kw)
    pi, pw = moe.route(part, 1, False, **kw)
    assert _repeats(ids, pi) and _repeats(w, pw)
    del ids, w
    _free()


def test_route_and_slot_map_of_the_most_pairs():
    """2^31 - 1 pairs: the last index is the last that 31 bits hold."""
    dev = device()
    _need(60)
    T = 2 ** 31 - 1
    announce(f"route and slot map T={T}")
    part = torch.randn(PERIOD, 1, generator=torch.Generator().manual_seed(6)).to(dev)
    logits = _repeat(part, T)
    ids, w = moe.route(logits, 1, False)
    del logits
    assert not ids.any() and bool((w == 1).all())
    w.view(-1)[-1] = 0.5
    slot, wm, mask = moe.slot_map(ids, w, 1)
    assert not slot.any() and torch.equal(wm, w) and bool((mask == 1).all())
    del ids, w, slot, wm, mask
    _free()


def test_combine():
    dev = device()
    _need(16)
    T, H = 2 ** 26 + 5, 8
    announce(f"combine T={T}")
    g = torch.Generator().manual_seed(2)
    y = torch.randn(PERIOD, H, generator=g).bfloat16().to(dev)
    rows = torch.randperm(PERIOD, generator=g).int().to(dev)
    wt = torch.rand(PERIOD, generator=g).to(dev)
    out = moe.combine(y, _repeat(rows, T), _repeat(wt, T), 1)
    assert _repeats(out, moe.combine(y, rows, wt, 1))
    del out
    _free()


@pytest.mark.parametrize("scaled", [False, True])
def test_permute(scaled):
    """The gathered rows of 2^24 + 5 tokens (a block of 256 threads each), all in one slot."""
    dev = device()
    _need(8)
    T, H = 2 ** 24 + 5, 8
    announce(f"permute T={T} scaled={scaled}")
    g = torch.Generator().manual_seed(3)
    x = torch.randn(PERIOD, H, generator=g).bfloat16().to(dev)
    wt = torch.rand(PERIOD, 1, generator=g).to(dev)
    slot = torch.zeros(T, 1, dtype=torch.int32, device=dev)
    mask = torch.ones(T, 1, dtype=torch.uint8, device=dev)
    off, pairs, row, xp = moe.permute(_repeat(x, T), slot, mask, 1, pair_w=_repeat(wt, T) if scaled else None)
    assert off.tolist() == [0, T]
    assert torch.equal(pairs, torch.arange(T, dtype=torch.int32, device=dev)) and torch.equal(row, pairs)
    assert _repeats(xp, (x.float() * wt).bfloat16() if scaled else x)
    del xp
    _free()


def test_layer_mxfp4():
    """2^26 + 3 tokens through one 4-bit expert: routing, permutation, products and combine."""
    dev = device()
    _need(60)
    T, H = 2 ** 26 + 3, 32
    announce(f"mxfp4 layer T={T}")
    g = torch.Generator().manual_seed(4)
    x = torch.randn(PERIOD, H, generator=g).bfloat16().to(dev)
    byte = lambda *s: torch.randint(0, 256, s, generator=g, dtype=torch.uint8).to(dev)  # noqa: E731
    gu, wd = byte(1, 64, 16), byte(1, 32, 16)
    gs, ds = (torch.full((1, n, 1), 125, dtype=torch.uint8, device=dev) for n in (64, 32))
    logits = torch.randn(PERIOD, 1, generator=g).to(dev)

    def layer(x, logits):
        cfg = moe.ForwardConfig(T=x.shape[0], H=H, I=32, E_global=1, K=1, renormalize=False, S=1, dtype=moe.MXFP4)
        return moe.forward(cfg, x, gu, wd, logits=logits, w_gate_up_scale=gs, w_down_scale=ds)
    assert _repeats(layer(_repeat(x, T), _repeat(logits, T)), layer(x, logits))
    _free()


def test_quantize_fp8():
    dev = device()
    _need(200)
    n, period = 2 ** 36 + 32, 16 * 4099
    announce(f"quantize fp8 n={n}")
    part = torch.randn(period, generator=torch.Generator().manual_seed(5)).bfloat16().to(dev)
    x = _repeat(part, n)
    q = moe.quantize_fp8(x, 0.01)
    del x
    assert _repeats(q, moe.quantize_fp8(part, 0.01))
    del q
    _free()
