"""What the operators around the fused MoE layer cost: the norm that feeds it, its router's loss and
gradient, and its experts with 4-bit weights.

Where `own` is false, run() computes an operator in its plain form with elementary torch operations in
32 bits; where it is true, run() makes the calls of this repository's package. Sizes are those of the
workloads in workloads/configs.py (hidden sizes, expert widths, expert counts, top-K) at the token
counts of decoding, of a chunk of a prompt, and of a training step.
"""
import math

import torch

own = False

MX_GROUP = 32          # weights that share one scale byte
FP8_MAX = 448.0
_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
_DT = {"f32": torch.float32, "bf16": torch.bfloat16}
_SIZE = {"f32": 4, "bf16": 2}


def listed():
    return [
        # one token of the 4096-wide layer between two layers of a decoding step, codes for FP8 experts
        {"name": "norm_token", "op": "norm", "T": 1, "H": 4096, "dtype": "bf16", "residual": True, "codes": True},
        # an f32 layer: an odd number of rows of an odd width, no residual and no codes
        {"name": "norm_f32", "op": "norm", "T": 777, "H": 2056, "dtype": "f32", "residual": False, "codes": False},
        # a whole prompt chunk before the 160-expert FP8 layer
        {"name": "norm_prefill", "op": "norm", "T": 8192, "H": 5120, "dtype": "bf16", "residual": True, "codes": True},
        # the smallest training step: 8 experts, top-2, all tokens valid
        {"name": "router_small", "op": "router", "T": 64, "E": 8, "K": 2, "renormalize": True, "pad": 0.0},
        # 60 experts, top-4, weights not renormalised, a padded batch
        {"name": "router_padded", "op": "router", "T": 4096, "E": 60, "K": 4, "renormalize": False, "pad": 0.2},
        # a large micro-batch of the 256-expert layer
        {"name": "router_large", "op": "router", "T": 65536, "E": 256, "K": 8, "renormalize": True, "pad": 0.0},
        # a single token through 60 experts of 1408, with the shared expert's output
        {"name": "experts_token", "op": "experts", "T": 1, "H": 2048, "I": 1408, "E": 60, "K": 4, "extra": 0, "ep": 1,
         "shared": True},
        # a decoding batch over 64 experts in 80 slots
        {"name": "experts_batch", "op": "experts", "T": 16, "H": 4096, "I": 1024, "E": 64, "K": 8, "extra": 16, "ep": 1,
         "shared": False},
        # one of four expert-parallel shares of 256 narrow experts: most slots hold one row or none
        {"name": "experts_share", "op": "experts", "T": 64, "H": 2048, "I": 512, "E": 256, "K": 8, "extra": 0, "ep": 4,
         "shared": False},
        # a chunk of a prompt: about 200 rows a slot, bound by arithmetic and no longer by the weights
        {"name": "experts_prompt", "op": "experts", "T": 2048, "H": 4096, "I": 1024, "E": 64, "K": 8, "extra": 16, "ep": 1,
         "shared": False},
        # one expert's stacked gate and up rows, quantised as a checkpoint is read, and read back
        {"name": "weights_expert", "op": "weights", "rows": 2816, "Kd": 2048, "dtype": "f32"},
        # the gate and up weights of a whole 64-expert layer
        {"name": "weights_layer", "op": "weights", "rows": 131072, "Kd": 4096, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("norm", "router", "experts", "experts", "weights"))
    if op == "norm":
        H = 8 * _log(rng, 32, 1024)
        dtype = rng.choice(("bf16", "bf16", "f32"))
        return {"op": op, "T": _log(rng, 1, min(16384, 16384 * 5120 // (H * _SIZE[dtype]))), "H": H, "dtype": dtype,
                "residual": rng.random() < 0.7, "codes": rng.random() < 0.7}
    if op == "router":
        E = _log(rng, 4, 256)
        return {"op": op, "T": _log(rng, 1, 65536), "E": E, "K": rng.randint(1, min(8, E)),
                "renormalize": rng.random() < 0.5, "pad": rng.choice((0.0, round(rng.random(), 3)))}
    if op == "experts":
        H, I = 32 * _log(rng, 8, 160), 32 * _log(rng, 4, 48)
        ep = rng.choice((1, 1, 2, 4))
        E = ep * _log(rng, 4, 160 // ep)
        K = rng.randint(1, min(8, E))
        return {"op": op, "T": min(_log(rng, 1, 2048), 2048 * 4096 * 1024 * 8 // (H * I * K)), "H": H, "I": I, "E": E, "K": K,
                "extra": rng.randint(0, E // ep // 4), "ep": ep, "shared": rng.random() < 0.3}
    rows = _log(rng, 1, 65536)
    return {"op": op, "rows": rows, "Kd": 32 * _log(rng, 2, 128), "dtype": rng.choice(("f32", "bf16"))}


# ---------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _mx_weights(g, S, N, Kd):
    """Codes and scales of weights about as wide as 1/sqrt(Kd): every code equally often, the groups'
    scales within a factor of four."""
    codes = torch.randint(0, 256, (S, N, Kd // 2), generator=g, device="cuda", dtype=torch.uint8)
    mid = 127 - 1 - int(round(0.5 * math.log2(Kd)))
    scale = torch.randint(mid - 1, mid + 1, (S, N, Kd // MX_GROUP), generator=g, device="cuda", dtype=torch.uint8)
    return codes, scale


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": case}
    if case["op"] == "norm":
        T, H, dt = case["T"], case["H"], _DT[case["dtype"]]
        s["x"] = _randn(g, T, H).to(dt)
        # the residual stream is wider than one layer's addition and has a few large channels
        wide = 1.0 + 20.0 * (torch.rand(H, generator=g, device="cuda") < 0.005)
        s["residual"] = (3.0 * wide * _randn(g, T, H)).to(dt) if case["residual"] else None
        s["gamma"] = (1.0 + 0.1 * _randn(g, H)).to(dt)
        s["eps"] = 1e-6
        s["scale"] = 1.0 / 56.0 if case["codes"] else None
    elif case["op"] == "router":
        T, E, K = case["T"], case["E"], case["K"]
        s["logits"] = _randn(g, T, E) + 0.5 * _randn(g, E)
        s["ids"] = torch.sort(s["logits"], dim=1, descending=True, stable=True)[1][:, :K].to(torch.int32).contiguous()
        s["dw"] = 1e-2 * _randn(g, T, K)
        s["coef"] = 1e-2
        s["mask"] = None
        if case["pad"]:
            # eight sequences padded to one length: the last part of each holds nothing
            rows = max(1, T // 8)
            at = torch.arange(T, device="cuda")
            empty = 2 * case["pad"] * torch.rand(T // rows + 1, generator=g, device="cuda")
            s["mask"] = (at % rows < ((1.0 - empty) * rows)[at // rows]).to(torch.uint8)
    elif case["op"] == "experts":
        T, H, I, E, ep = case["T"], case["H"], case["I"], case["E"], case["ep"]
        El, extra = E // ep, case["extra"]
        s["x"] = _randn(g, T, H).to(torch.bfloat16)
        s["logits"] = _randn(g, T, E)
        s["rank"] = ep - 1
        gu = _mx_weights(g, El, 2 * I, H)
        down = _mx_weights(g, El, H, I)
        # the first `extra` local experts hold a second slot with a copy of their weights
        own_slots = torch.arange(El, device="cuda")
        held = torch.cat([own_slots, own_slots[:extra]])
        s["gate_up"], s["gate_up_scale"] = (t[held].contiguous() for t in gu) if extra else gu
        s["down"], s["down_scale"] = (t[held].contiguous() for t in down) if extra else down
        count = 1 + (own_slots < extra).to(torch.int32)
        s["rep_off"] = torch.cat([torch.zeros(1, device="cuda"), count.cumsum(0)]).to(torch.int32)
        s["rep_slots"] = torch.sort(held, stable=True)[1].to(torch.int32)
        s["shared"] = _randn(g, T, H).to(torch.bfloat16) if case["shared"] else None
    else:
        w = _randn(g, case["rows"], case["Kd"])
        # groups of different widths, as rows and channels of trained weights are
        w *= 0.02 * torch.exp(0.5 * _randn(g, case["rows"], 1))
        s["w"] = w.to(_DT[case["dtype"]])
    return s


# ---------------------------------------------------------------- plain forms
def _norm_plain(s):
    x = s["x"]
    h = x.float() + s["residual"].float() if s["residual"] is not None else x.float()
    v = h * (h.square().mean(1, keepdim=True) + s["eps"]).rsqrt() * s["gamma"].float()
    out = {"y": v.to(x.dtype)}
    if s["residual"] is not None:
        out["residual"] = h.to(x.dtype)
    if s["scale"] is not None:
        out["codes"] = (v * (1.0 / s["scale"])).clamp(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn)
    return out


def _router_plain(s):
    logits, K, E = s["logits"], s["case"]["K"], s["case"]["E"]
    ids, dw = s["ids"].long(), s["dw"]
    valid = torch.ones_like(logits[:, :1], dtype=torch.bool) if s["mask"] is None else s["mask"][:, None] != 0
    e = (logits - logits.amax(1, keepdim=True)).exp()
    p = torch.where(valid, e / e.sum(1, keepdim=True), 0.0)
    n = valid.sum()
    counts = torch.zeros(E, dtype=torch.int32, device=logits.device)
    counts.scatter_add_(0, ids.flatten(), valid.expand(-1, K).flatten().to(torch.int32))
    share = 1.0 / n.clamp(min=1).float()
    prob = p.sum(0) * share
    f = counts.float() * (share / K)
    loss = s["coef"] * E * (f * prob).sum()
    ps = p.gather(1, ids)
    if s["case"]["renormalize"]:
        w = ps / ps.sum(1, keepdim=True)
        d = torch.zeros_like(p).scatter_add_(1, ids, w * (dw - (w * dw).sum(1, keepdim=True)))
    else:
        d = (-p * (ps * dw).sum(1, keepdim=True)).scatter_add_(1, ids, ps * dw)
    d = d + s["coef"] * E * share * p * (f - (p * f).sum(1, keepdim=True))
    return {"loss": loss, "counts": torch.cat([counts, n[None].to(torch.int32)]), "prob": prob,
            "dlogits": torch.where(valid, d, 0.0)}


def _mx_values(codes, scale, dt=torch.float32):
    """The weights that codes [..., K/2] and scales [..., K/32] stand for, as [..., K]."""
    table = torch.tensor(_E2M1 + tuple(-v for v in _E2M1), dtype=dt, device=codes.device)
    both = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
    v = table[both.int()].unflatten(-1, (-1, MX_GROUP))
    return (v * torch.exp2(scale.to(dt) - 127.0)[..., None]).flatten(-2)


def _routed(s):
    """(slot, weight) of every pair; the weight of a pair of another rank is 0."""
    c = s["case"]
    El = c["E"] // c["ep"]
    e = (s["logits"] - s["logits"].amax(1, keepdim=True)).exp()
    p = e / e.sum(1, keepdim=True)
    ids = torch.sort(s["logits"], dim=1, descending=True, stable=True)[1][:, :c["K"]]
    w = p.gather(1, ids)
    w = w / w.sum(1, keepdim=True)
    lid = ids - s["rank"] * El
    local = (lid >= 0) & (lid < El)
    lid = lid.clamp(0, El - 1)
    first, last = s["rep_off"].long()[lid], s["rep_off"].long()[lid + 1]
    t = torch.arange(c["T"], device=ids.device)[:, None]
    return s["rep_slots"].long()[first + t % (last - first)], torch.where(local, w, 0.0)


def _experts_plain(s):
    c = s["case"]
    T, K, I, S = c["T"], c["K"], c["I"], s["gate_up"].shape[0]
    slot, w = _routed(s)
    x = s["x"].float()
    if T * K < S:  # fewer pairs than slots: each pair's own weights
        at = slot.flatten()
        h = x.repeat_interleave(K, 0)[:, None] @ _mx_values(s["gate_up"][at], s["gate_up_scale"][at]).transpose(1, 2)
        a = h[..., :I] / (1.0 + (-h[..., :I]).exp()) * h[..., I:]
        y = a @ _mx_values(s["down"][at], s["down_scale"][at]).transpose(1, 2)
        out = (y[:, 0].unflatten(0, (T, K)) * w[..., None]).sum(1)
    else:          # every slot's weights once, every token through them, weight 0 where it does not belong
        by_slot = torch.zeros(T, S, device=x.device).scatter_add_(1, slot, w)
        h = x @ _mx_values(s["gate_up"], s["gate_up_scale"]).transpose(1, 2)
        a = h[..., :I] / (1.0 + (-h[..., :I]).exp()) * h[..., I:]
        a = a * by_slot.t()[..., None]
        out = (a @ _mx_values(s["down"], s["down_scale"]).transpose(1, 2)).sum(0)
    if s["shared"] is not None:
        out = out + s["shared"].float()
    return {"out": out.to(torch.bfloat16)}


def _weights_plain(s):
    w = s["w"].float().unflatten(-1, (-1, MX_GROUP))
    _, e = torch.frexp(w.abs().amax(-1, keepdim=True))  # amax in [2^(e-1), 2^e)
    b = (e + (127 - 3)).clamp(0, 254)
    v = w * torch.exp2((127 - b).float())
    a = v.abs()
    code = ((a > 0.25).to(torch.int32) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    value = torch.tensor(_E2M1, device=w.device)[code].copysign(v) * torch.exp2((b - 127).float())
    return {"values": value.flatten(-2).to(torch.bfloat16)}


# ---------------------------------------------------------------- one pass
def _norm_own(s):
    import moe_expert_dispatch_amd as moe
    y, residual, q = moe.rms_norm(s["x"], s["gamma"], s["eps"], residual=s["residual"], q_scale=s["scale"])
    out = {"y": y}
    if s["residual"] is not None:
        out["residual"] = residual
    if s["scale"] is not None:
        out["codes"] = q.view(torch.float8_e4m3fn)
    return out


def _router_own(s):
    import moe_expert_dispatch_amd as moe
    loss, counts, prob = moe.balance_loss(s["logits"], s["ids"], s["coef"], token_mask=s["mask"])
    d = moe.route_backward(s["logits"], s["ids"], s["dw"], s["case"]["renormalize"], counts=counts, coef=s["coef"],
                           token_mask=s["mask"])
    return {"loss": loss, "counts": counts, "prob": prob, "dlogits": d}


def _experts_own(s):
    import moe_expert_dispatch_amd as moe
    c = s["case"]
    cfg = moe.ForwardConfig(T=c["T"], H=c["H"], I=c["I"], E_global=c["E"], K=c["K"], renormalize=True,
                            S=s["gate_up"].shape[0], dtype=moe.MXFP4, ep_size=c["ep"], ep_rank=s["rank"])
    out = moe.forward(cfg, s["x"], s["gate_up"], s["down"], logits=s["logits"], rep_off=s["rep_off"],
                      rep_slots=s["rep_slots"], shared_out=s["shared"], w_gate_up_scale=s["gate_up_scale"],
                      w_down_scale=s["down_scale"])
    return {"out": out}


def _weights_own(s):
    import moe_expert_dispatch_amd as moe
    codes, scale = moe.quantize_mxfp4(s["w"])
    return {"values": moe.dequantize_mxfp4(codes, scale, torch.bfloat16)}


def run(state):
    op = state["case"]["op"]
    if own:
        return {"norm": _norm_own, "router": _router_own, "experts": _experts_own, "weights": _weights_own}[op](state)
    return {"norm": _norm_plain, "router": _router_plain, "experts": _experts_plain, "weights": _weights_plain}[op](state)


# ---------------------------------------------------------------- least work
def work(case):
    if case["op"] == "norm":
        b = _SIZE[case["dtype"]]
        n = case["T"] * case["H"]
        return {"bytes": n * (2 * b + (2 * b if case["residual"] else 0) + (1 if case["codes"] else 0)) + case["H"] * b,
                "flops": 6 * n}
    if case["op"] == "router":
        T, E, K = case["T"], case["E"], case["K"]
        return {"bytes": 8 * T * E + 8 * T * K + (T if case["pad"] else 0) + 8 * E, "flops": 16 * T * E}
    if case["op"] == "experts":
        T, H, I, E, K, ep = (case[k] for k in ("T", "H", "I", "E", "K", "ep"))
        # slots that some token reaches, for tokens that choose K of E evenly; a second slot takes half of its expert's
        some = 1 - (1 - K / E) ** T
        half = 1 - (1 - 0.5 * K / E) ** T
        slots = (E // ep - case["extra"]) * some + 2 * case["extra"] * half
        weights = slots * 3 * H * I * 17 / 32
        return {"bytes": weights + T * H * (6 if case["shared"] else 4) + T * E * 4, "flops": 6 * H * I * T * K / ep}
    n = case["rows"] * case["Kd"]
    return {"bytes": n * (_SIZE[case["dtype"]] + 2 * 17 / 32 + 2), "flops": 4 * n}


# ---------------------------------------------------------------- 64 bits
def _norm_exact(s):
    h = s["x"].double()
    if s["residual"] is not None:
        h = h + s["residual"].double()
    norm = torch.linalg.vector_norm(h, dim=1, keepdim=True)
    v = h / torch.sqrt(norm * norm / h.shape[1] + s["eps"]) * s["gamma"].double()
    out = {"y": v}
    if s["residual"] is not None:
        out["residual"] = h
    if s["scale"] is not None:  # before its rounding, as y
        out["codes"] = torch.clamp(v / s["scale"], -FP8_MAX, FP8_MAX)
    return out


def _router_exact(s):
    c = s["case"]
    T, E, K = c["T"], c["E"], c["K"]
    keep = torch.arange(T, device="cuda") if s["mask"] is None else torch.nonzero(s["mask"]).flatten()
    n = keep.numel()
    out = {"loss": torch.zeros((), dtype=torch.float64), "counts": None, "prob": torch.zeros(E, dtype=torch.float64),
           "dlogits": torch.zeros(T, E, dtype=torch.float64, device="cuda")}
    if n == 0:
        return out
    l = s["logits"][keep].double()
    p = torch.softmax(l, 1)
    chosen = torch.nn.functional.one_hot(s["ids"][keep].long(), E).double()  # [n, K, E]
    f = chosen.sum((0, 1)) / (n * K)
    prob = p.mean(0)
    # dL/dp, then through the softmax's Jacobian
    up = s["dw"][keep].double()
    if c["renormalize"]:
        ps = (chosen * p[:, None]).sum(2)
        total = ps.sum(1, keepdim=True)
        up = up / total - (up * ps).sum(1, keepdim=True) / total ** 2
    dp = (chosen * up[..., None]).sum(1) + s["coef"] * E / n * f
    out["dlogits"][keep] = p * (dp - (p * dp).sum(1, keepdim=True))
    out["loss"], out["prob"] = s["coef"] * E * torch.dot(f, prob), prob
    return out


def _mx_decoded(codes, scale):
    """One matrix in 64 bits, from the format's fields: sign, two bits of exponent, one of mantissa."""
    out = torch.empty(codes.shape[0], 2 * codes.shape[1], dtype=torch.float64, device=codes.device)
    for half in (0, 1):
        c = (codes >> (4 * half)) & 15
        e, m = (c >> 1) & 3, (c & 1).double()
        mag = torch.where(e == 0, 0.5 * m, torch.ldexp(1.0 + 0.5 * m, e.double() - 1.0))
        out[:, half::2] = torch.where(c >= 8, -mag, mag)
    return out * torch.ldexp(torch.ones_like(scale, dtype=torch.float64), scale.double() - 127.0).repeat_interleave(
        MX_GROUP, 1)


def _experts_exact(s):
    c = s["case"]
    T, H, I, E, K = (c[k] for k in ("T", "H", "I", "E", "K"))
    El = E // c["ep"]
    l = s["logits"].double().cpu()
    out = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    if s["shared"] is not None:
        out += s["shared"].double()
    rows = {}
    for t in range(T):  # the token's K largest logits, their weights, the slots that hold them
        best = torch.sort(l[t], descending=True, stable=True)[1][:K]
        w = torch.softmax(l[t][best], 0)
        for e, v in zip(best.tolist(), w.tolist()):
            e -= s["rank"] * El
            if 0 <= e < El:
                rows.setdefault(El + e if e < c["extra"] and t % 2 else e, []).append((t, v))
    for slot, pairs in rows.items():
        at = torch.tensor([t for t, _ in pairs], device="cuda")
        w = torch.tensor([v for _, v in pairs], dtype=torch.float64, device="cuda")
        h = s["x"][at].double() @ _mx_decoded(s["gate_up"][slot], s["gate_up_scale"][slot]).t()
        a = h[:, :I] * torch.sigmoid(h[:, :I]) * h[:, I:]
        y = a @ _mx_decoded(s["down"][slot], s["down_scale"][slot]).t()
        out[at] += w[:, None] * y
    return {"out": out}


def _weights_exact(s):
    w = s["w"].double().unflatten(-1, (-1, MX_GROUP))
    top = w.abs().amax(-1, keepdim=True)
    unit = torch.exp2(torch.floor(torch.log2(torch.where(top > 0, top, 1.0))) - 2)
    a = (w / unit).abs()
    # steps of 0.5 below 2, of 1 below 4, of 2 above; halves to the even multiple
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0)).to(a.dtype)
    return {"values": (torch.clamp(torch.round(a / step) * step, max=6.0).copysign(w) * unit).flatten(-2)}


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _norm_exact, "router": _router_exact, "experts": _experts_exact, "weights": _weights_exact}[
        case["op"]](s)
