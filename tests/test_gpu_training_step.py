"""A whole training step of the layer, norm to loss and back, from the library's calls: against the fp64
gradient that torch forms of the same layer with the same routing, captured in a graph, and on two streams.

Tolerance of the f32 step, on the 2-norm of each gradient: eight products follow one another, each of at most
n = 136 terms with an error of at most 2 n u of its terms' magnitudes, u = 2^-24; for terms of random signs
these are some sqrt(n) times the result, so 8 * 2 * 136 * 12 u = 1.6e-3 at the very most. A wrong term, weight
or row is of the gradient's own size.
"""
import numpy as np
import pytest
import torch

import moe_expert_dispatch_amd as moe
from gpu_common import announce, device, rel_fro

pytestmark = pytest.mark.gpu

F32_STEP = 1.6e-3


class Layer:
    """E experts in S slots, the first `extra` of them in two."""

    def __init__(self, T, H, I, E, K, extra, seed, dt, dev):
        g = torch.Generator().manual_seed(seed)
        n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
        self.T, self.H, self.I, self.E, self.K, self.S, self.dt = T, H, I, E, K, E + extra, dt
        put = lambda t: t.to(dt).to(dev)  # noqa: E731
        self.x, self.res, self.dout = put(n(T, H)), put(n(T, H)), put(n(T, H))
        self.dres_out = put(n(T, H) * 0.3)
        self.gamma, self.beta = put(1 + 0.2 * n(H)), put(0.2 * n(H))
        self.router = (n(E, H) / H ** 0.5).to(dev)
        self.gu, self.wd = put(n(E, 2 * I, H) / H ** 0.5), put(n(E, H, I) / I ** 0.5)
        held = torch.cat([torch.arange(E), torch.arange(extra)])
        self.held = held.to(dev)
        count = 1 + (torch.arange(E) < extra).int()
        self.rep_off = torch.cat([torch.zeros(1), count.cumsum(0)]).int().to(dev)
        self.rep_slots = torch.sort(held, stable=True)[1].int().to(dev)
        self.coef = 0.05

    def step(self):
        """Forward and backward pass; every gradient."""
        K, S = self.K, self.S
        gu, wd = self.gu[self.held], self.wd[self.held]   # the slots' copies
        y, r, _ = moe.layer_norm(self.x, self.gamma, self.beta, 1e-5, residual=self.res)
        logits = y.float() @ self.router.t()
        ids, w = moe.route(logits, K, True)
        loss, counts, _ = moe.balance_loss(logits, ids, self.coef)
        slot, wm, mask = moe.slot_map(ids, w, self.E, rep_off=self.rep_off, rep_slots=self.rep_slots)
        off, _, rows, xp = moe.permute(y, slot, mask, S)
        h = moe.grouped_gemm(moe.DOWN, xp, off, gu)
        act = moe.swiglu(h, off)
        ye = moe.grouped_gemm(moe.DOWN, act, off, wd)
        out = moe.combine(ye, rows, wm, K, shared=r)      # the residual stream beside the experts

        dye, dw = moe.combine_backward(self.dout, ye, rows, wm, K)
        dh = moe.grouped_gemm_backward(moe.DOWN, dye, off, wd, h=h)
        dxp = moe.grouped_gemm_backward(moe.GATE_UP_SWIGLU, dh, off, gu)
        dwd = moe.grouped_gemm_weight_grad(dye, act, off)
        dgu = moe.grouped_gemm_weight_grad(dh, xp, off)
        dlogits = moe.route_backward(logits, ids, dw, True, counts=counts, coef=self.coef)
        dy = dlogits @ self.router                        # f32; the experts' part is added to it
        dy, _ = moe.permute_backward(dxp, rows, K, dx=dy, accumulate=True)
        dstream = (self.dout.float() + self.dres_out.float()).to(self.dt)
        dx, dgamma, dbeta = moe.layer_norm_backward(dy.to(self.dt), r, self.gamma, 1e-5, dresidual=dstream)
        fold = lambda t: torch.zeros(self.E, *t.shape[1:], device=t.device).index_add_(0, self.held, t)  # noqa: E731
        return {"out": out, "loss": loss, "dx": dx, "dgamma": dgamma, "dbeta": dbeta, "dgu": fold(dgu), "dwd": fold(dwd),
                "drouter": dlogits.t() @ y.float()}, ids

    def reference(self, ids):
        """The same in fp64 by differentiation; counts are constants of the loss."""
        c = lambda t: t.detach().double().cpu()  # noqa: E731
        x, res, gamma, beta, gu, wd, router = (c(t).requires_grad_() for t in
                                               (self.x, self.res, self.gamma, self.beta, self.gu, self.wd, self.router))
        ids = ids.cpu().long()
        r = x + res
        var, mean = torch.var_mean(r, 1, correction=0, keepdim=True)
        y = (r - mean) / torch.sqrt(var + 1e-5) * gamma + beta
        p = torch.softmax(y @ router.t(), 1)
        ps = p.gather(1, ids)
        w = ps / ps.sum(1, keepdim=True)
        f = torch.bincount(ids.flatten(), minlength=self.E).double() / ids.numel()
        loss = self.coef * self.E * (f * p.mean(0)).sum()
        out = r.clone()
        for e in range(self.E):
            t, k = torch.nonzero(ids == e, as_tuple=True)
            h = y[t] @ gu[e].t()
            act = torch.nn.functional.silu(h[:, :self.I]) * h[:, self.I:]
            out = out.index_add(0, t, w[t, k][:, None] * (act @ wd[e].t()))
        total = (out * c(self.dout)).sum() + (r * c(self.dres_out)).sum() + loss
        got = torch.autograd.grad(total, (x, gamma, beta, gu, wd, router))
        names = ("dx", "dgamma", "dbeta", "dgu", "dwd", "drouter")
        return {"out": out.detach(), "loss": loss.detach(), **dict(zip(names, got))}


@pytest.mark.parametrize("T,H,I,E,K,extra", [(1, 64, 40, 4, 2, 0), (37, 136, 72, 6, 3, 2), (300, 128, 64, 16, 4, 4),
                                             (64, 72, 136, 3, 3, 3)])
def test_step_in_f32_against_differentiation(T, H, I, E, K, extra):
    dev = device()
    announce(f"training step f32 T={T} H={H} I={I} E={E} K={K}")
    L = Layer(T, H, I, E, K, extra, T + H, torch.float32, dev)
    got, ids = L.step()
    want = L.reference(ids)
    for k in want:
        assert rel_fro(got[k].double().cpu().numpy(), want[k].numpy()) < F32_STEP, k


def test_step_in_bf16_against_differentiation():
    """bf16 between the stages: some ten roundings of 2^-8 at most follow one another, each of them spread
    over a sum, so a gradient is within 10 * 2^-8 of the one of the same bf16 inputs, on the 2-norm."""
    dev = device()
    announce("training step bf16")
    L = Layer(500, 256, 128, 12, 4, 3, 11, torch.bfloat16, dev)
    got, ids = L.step()
    want = L.reference(ids)
    for k in want:
        assert rel_fro(got[k].double().cpu().numpy(), want[k].numpy()) < 10 * 2.0 ** -8, k


@pytest.mark.parametrize("dt,T", [(torch.bfloat16, 3), (torch.bfloat16, 700), (torch.float32, 90), (torch.bfloat16, 20000)])
def test_step_captured_in_a_graph_and_on_two_streams(dt, T):
    """Captured once, replayed on new inputs with eager steps between; then two steps at once on two streams."""
    dev = device()
    announce(f"training step graph {dt} T={T}")
    L = Layer(T, 128, 64, 6, 2, 2, 5, dt, dev)

    def step():
        # the library's calls alone, on given routing: torch's own sums over blocks are not at issue
        w = L.w
        slot, wm, mask = moe.slot_map(L.ids, w, L.E, rep_off=L.rep_off, rep_slots=L.rep_slots)
        y, r, _ = moe.layer_norm(L.x, L.gamma, L.beta, 1e-5, residual=L.res)
        off, _, rows, xp = moe.permute(y, slot, mask, L.S, pair_w=wm)
        h = moe.grouped_gemm(moe.DOWN, xp, off, L.slots[0])
        act = moe.swiglu(h, off)
        ye = moe.grouped_gemm(moe.DOWN, act, off, L.slots[1])
        dye, dw = moe.combine_backward(L.dout, ye, rows, wm, L.K)
        dh = moe.grouped_gemm_backward(moe.DOWN, dye, off, L.slots[1], h=h)
        dxp = moe.grouped_gemm_backward(moe.GATE_UP_SWIGLU, dh, off, L.slots[0])
        dwd = moe.grouped_gemm_weight_grad(dye, act, off)
        dgu = moe.grouped_gemm_weight_grad(dh, xp, off, dw_dtype=dt)
        dx, dpw = moe.permute_backward(dxp, rows, L.K, wm, y)
        return (*moe.layer_norm_backward(dx, r, L.gamma, 1e-5, dresidual=L.dres_out),
                *moe.rms_norm_backward(dx, r, L.gamma, 1e-5), dw, dpw, dwd, dgu)

    L.slots = (L.gu[L.held].contiguous(), L.wd[L.held].contiguous())

    def inputs(i):
        g = torch.Generator(device=dev).manual_seed(i)
        for t in (L.x, L.res, L.dout, L.dres_out):
            t.copy_(torch.randn(t.shape, generator=g, device=dev))
        return (torch.sort(torch.rand(T, L.E, generator=g, device=dev), 1)[1][:, :L.K].int().contiguous(),
                torch.rand(T, L.K, generator=g, device=dev))

    L.ids, L.w = inputs(99)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for i in range(4):
        ids, w = inputs(i)
        L.ids.copy_(ids)
        L.w.copy_(w)
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in outs]
        for a, b in zip(got, step()):
            assert torch.equal(a, b), i
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
    for o in outs:
        assert all(torch.equal(a, b) for a, b in zip(o, want))
