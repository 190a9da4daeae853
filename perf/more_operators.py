"""What the training pass of the MoE layer costs: layer norm forward and backward, the gradients of the
permutation and of the weighted sum back into token order, and the gradients of the experts' products.

Where `own` is false, run() computes an operator in its plain form with elementary torch operations in
32 bits; where it is true, run() makes the calls of this repository's package. Sizes are those of the
workloads in workloads/configs.py (hidden sizes, expert widths, expert counts, top-K) at token counts from
a small batch to a large micro-batch of a training step.
"""
import math

import torch

own = False

_DT = {"f32": torch.float32, "bf16": torch.bfloat16}
_SIZE = {"f32": 4, "bf16": 2}


def listed():
    return [
        # a small batch before the 60-expert layer: latency counts
        {"name": "norm_small", "op": "norm", "kind": "layer", "T": 64, "H": 2048, "dtype": "bf16", "residual": False},
        # an f32 layer: an odd number of rows of an odd width, no residual
        {"name": "norm_f32", "op": "norm", "kind": "layer", "T": 777, "H": 2056, "dtype": "f32", "residual": False},
        # a large micro-batch, the residual stream's addition and its gradient with it
        {"name": "norm_large", "op": "norm", "kind": "layer", "T": 16384, "H": 4096, "dtype": "bf16", "residual": True},
        # the gradient of the RMS norm before the 160-expert layer, with the residual stream's
        {"name": "norm_rms", "op": "norm", "kind": "rms", "T": 8192, "H": 5120, "dtype": "bf16", "residual": True},
        # the smallest step of the 60-expert layer
        {"name": "rows_small", "op": "rows", "T": 64, "H": 2048, "E": 60, "K": 4, "ep": 1, "on_input": False, "dtype": "bf16"},
        # weights applied on the experts' input, one of four expert-parallel shares, an odd batch in f32
        {"name": "rows_input", "op": "rows", "T": 1999, "H": 2056, "E": 256, "K": 8, "ep": 4, "on_input": True, "dtype": "f32"},
        # the 64-expert layer's micro-batch: every pair local
        {"name": "rows_large", "op": "rows", "T": 16384, "H": 4096, "E": 64, "K": 8, "ep": 1, "on_input": False, "dtype": "bf16"},
        # the f32 layer of 8 experts: an odd batch of odd widths
        {"name": "experts_f32", "op": "experts", "T": 333, "H": 264, "I": 136, "E": 8, "K": 2, "dtype": "f32"},
        # a few rows for each of 60 experts: bound by reading and writing the weights
        {"name": "experts_few", "op": "experts", "T": 128, "H": 2048, "I": 1408, "E": 60, "K": 4, "dtype": "bf16"},
        # a micro-batch of the 64-expert layer, bound by arithmetic
        {"name": "experts_large", "op": "experts", "T": 4096, "H": 4096, "I": 1024, "E": 64, "K": 8, "dtype": "bf16"},
        # narrow experts of an expert-parallel share: the down weights' gradient, f32 for an optimizer's sums
        {"name": "weights_narrow", "op": "weights", "T": 1024, "N": 2048, "Kd": 512, "E": 64, "K": 2, "dtype": "bf16"},
        # the gate and up weights' gradient of the large layer
        {"name": "weights_large", "op": "weights", "T": 16384, "N": 2048, "Kd": 4096, "E": 64, "K": 8, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("norm", "norm", "rows", "experts", "weights"))
    if op == "norm":
        H = 8 * _log(rng, 16, 1024)
        dtype = rng.choice(("bf16", "bf16", "f32"))
        return {"op": op, "kind": rng.choice(("layer", "rms")), "T": _log(rng, 1, min(65536, 16384 * 8192 // (H * _SIZE[dtype]))),
                "H": H, "dtype": dtype, "residual": rng.random() < 0.6}
    if op == "rows":
        H = 8 * _log(rng, 16, 1024)
        dtype = rng.choice(("bf16", "bf16", "f32"))
        ep = rng.choice((1, 1, 2, 4))
        E = ep * _log(rng, 4, 256 // ep)
        K = rng.randint(1, min(8, E))
        return {"op": op, "T": _log(rng, 1, min(32768, 16384 * 8192 * 8 // (H * K * _SIZE[dtype]))), "H": H, "E": E, "K": K, "ep": ep,
                "on_input": rng.random() < 0.4, "dtype": dtype}
    dtype = rng.choice(("bf16", "bf16", "bf16", "f32"))
    E = _log(rng, 4, 64)
    K = rng.randint(1, min(8, E))
    if op == "experts":
        most = 2048 if dtype == "bf16" else 512
        H, I = 8 * _log(rng, 16, most // 8), 8 * _log(rng, 8, most // 16)
        return {"op": op, "T": min(_log(rng, 1, 4096), 4096 * 1024 * 2048 // (H * I * K)), "H": H, "I": I, "E": E, "K": K, "dtype": dtype}
    most = 4096 if dtype == "bf16" else 512
    N, Kd = 8 * _log(rng, 16, most // 8), 8 * _log(rng, 16, most // 8)
    return {"op": op, "T": max(1, min(_log(rng, 1, 8192), 16384 * 4096 * 512 // (N * Kd * K // 8 + 1))), "N": N, "Kd": Kd, "E": E, "K": K,
            "dtype": dtype}


# ---------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _permutation(g, T, E, K, ep):
    """What moe.permute() gives for tokens routed by logits with a bias of each expert: the slots' row
    offsets, the pairs in the order of the rows, each pair's row or -1. The last rank's share."""
    ids = torch.sort(_randn(g, T, E) + 0.5 * _randn(g, E), dim=1, descending=True, stable=True)[1][:, :K]
    El = E // ep
    slot = (ids - (ep - 1) * El).flatten()
    local = slot >= 0
    order = torch.sort(torch.where(local, slot, El), stable=True)[1]
    counts = torch.zeros(El, dtype=torch.int64, device="cuda").scatter_add_(0, slot.clamp(min=0), local.long())
    offsets = torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), counts.cumsum(0)])
    rows = int(offsets[-1].item())
    pair_row = torch.full((T * K,), -1, dtype=torch.int32, device="cuda")
    pair_row[order[:rows]] = torch.arange(rows, dtype=torch.int32, device="cuda")
    return {"offsets": offsets.to(torch.int32), "sorted_pairs": order[:rows].to(torch.int32), "pair_row": pair_row, "rows": rows,
            "cap": int(counts.max().item())}


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": case}
    dt = _DT[case["dtype"]]
    if case["op"] == "norm":
        T, H = case["T"], case["H"]
        s["x"] = (_randn(g, T, H) + 0.3 * _randn(g, T, 1)).to(dt)
        # the residual stream is wider than one layer's addition and has a few large channels
        wide = 1.0 + 20.0 * (torch.rand(H, generator=g, device="cuda") < 0.005)
        s["residual"] = (3.0 * wide * _randn(g, T, H)).to(dt) if case["residual"] else None
        # the row that the forward pass kept, of the stream behind the addition
        s["kept"] = s["x"] if s["residual"] is None else (s["x"].float() + s["residual"].float()).to(dt)
        s["gamma"] = (1.0 + 0.1 * _randn(g, H)).to(dt)
        s["beta"] = (0.1 * _randn(g, H)).to(dt)
        s["dy"] = (1e-2 * _randn(g, T, H)).to(dt)
        s["dresidual"] = (1e-2 * _randn(g, T, H)).to(dt) if case["residual"] else None
        s["eps"] = 1e-5
        return s
    T, K = case["T"], case["K"]
    s.update(_permutation(g, T, case["E"], K, case.get("ep", 1)))
    P = s["rows"]
    if case["op"] == "rows":
        H = case["H"]
        w = torch.softmax(_randn(g, T, K), 1)
        s["w"] = torch.where(s["pair_row"].view(T, K) >= 0, w, 0.0)
        s["dout"] = (1e-2 * _randn(g, T, H)).to(dt)
        # rows for every pair, as the permutation has them; a share fills the first of them
        s["y"] = _randn(g, T * K, H).to(dt)
        s["x"] = _randn(g, T, H).to(dt) if case["on_input"] else None
        s["dx_perm"] = (1e-2 * _randn(g, T * K, H)).to(dt)
        s["dy"] = torch.zeros(T * K, H, dtype=dt, device="cuda")
    elif case["op"] == "experts":
        H, I, E = case["H"], case["I"], case["E"]
        s["w_gate_up"] = (_randn(g, E, 2 * I, H) / math.sqrt(H)).to(dt)
        s["w_down"] = (_randn(g, E, H, I) / math.sqrt(I)).to(dt)
        s["x_perm"] = _randn(g, P, H).to(dt)
        s["h"] = (1.2 * _randn(g, P, 2 * I)).to(dt)  # what the gate/up product gave
        s["dy"] = (1e-2 * _randn(g, P, H)).to(dt)
    else:
        s["dc"] = (1e-2 * _randn(g, P, case["N"])).to(dt)
        s["a"] = _randn(g, P, case["Kd"]).to(dt)
    return s


# ---------------------------------------------------------------- plain forms
def _norm_plain(s):
    dt, kind = s["x"].dtype, s["case"]["kind"]
    gamma, dy, out = s["gamma"].float(), s["dy"].float(), {}
    if kind == "layer":
        h = s["x"].float() + s["residual"].float() if s["residual"] is not None else s["x"].float()
        c = h - h.mean(1, keepdim=True)
        out["y"] = (c * (c.square().mean(1, keepdim=True) + s["eps"]).rsqrt() * gamma + s["beta"].float()).to(dt)
        if s["residual"] is not None:
            out["residual"] = h.to(dt)
    x = s["kept"].float()
    c = x - x.mean(1, keepdim=True) if kind == "layer" else x
    r = (c.square().mean(1, keepdim=True) + s["eps"]).rsqrt()
    n, d = c * r, dy * gamma
    dx = d - n * (d * n).mean(1, keepdim=True)
    if kind == "layer":
        dx = dx - d.mean(1, keepdim=True)
        out["dbeta"] = dy.sum(0)
    dx = dx * r
    if s["dresidual"] is not None:
        dx = dx + s["dresidual"].float()
    out["dx"] = dx.to(dt)
    out["dgamma"] = (dy * n).sum(0)
    return out


def _rows_plain(s):
    T, K = s["case"]["T"], s["case"]["K"]
    dt, on_input = s["dout"].dtype, s["case"]["on_input"]
    pairs = s["sorted_pairs"].long()
    row = s["pair_row"].long().clamp(min=0).view(T, K)
    local = (s["pair_row"] >= 0).view(T, K)
    d = s["dout"].float()[pairs // K]
    w = s["w"].flatten()
    out = {"dy": s["dy"]}
    if on_input:
        s["dy"][:s["rows"]] = d.to(dt)
    else:
        s["dy"][:s["rows"]] = (w[pairs][:, None] * d).to(dt)
        y = s["y"][:s["rows"]].float()
        out["dw"] = torch.zeros(T * K, device=d.device).index_copy_(0, pairs, (d * y).sum(1)).view(T, K)
    dxp = torch.where(local[..., None], s["dx_perm"].float()[row], 0.0)
    if on_input:
        out["dx"] = (dxp * s["w"][..., None]).sum(1).to(dt)
        out["dpair_w"] = (dxp * s["x"].float()[:, None]).sum(2)
    else:
        out["dx"] = dxp.sum(1).to(dt)
    return out


def _padded(s, *rows):
    """Rows [P, C] as [slots, cap, C] in 32 bits, zeros behind a slot's last, and the place of each row there."""
    off = s["offsets"].long()
    at = off[:-1, None] + torch.arange(s["cap"], device=off.device)
    inside = at < off[1:, None]
    return inside, [torch.where(inside[..., None], r.float()[at.clamp(max=s["rows"] - 1)], 0.0) for r in rows]


def _experts_plain(s):
    I, dt = s["case"]["I"], s["h"].dtype
    inside, (x, h, dy) = _padded(s, s["x_perm"], s["h"], s["dy"])
    g, u = h[..., :I], h[..., I:]
    sig = 1.0 / (1.0 + (-g).exp())
    act = g * sig * u
    da = dy @ s["w_down"].float()
    dh = torch.cat([da * u * sig * (1.0 + g * (1.0 - sig)), da * g * sig], -1)
    return {"act": act[inside].to(dt), "dh": dh[inside].to(dt), "dx": (dh @ s["w_gate_up"].float())[inside].to(dt),
            "dw_down": (dy.transpose(1, 2) @ act).to(dt), "dw_gate_up": (dh.transpose(1, 2) @ x).to(dt)}


def _weights_plain(s):
    _, (dc, a) = _padded(s, s["dc"], s["a"])
    return {"dw": dc.transpose(1, 2) @ a}


# ---------------------------------------------------------------- one pass
def _norm_own(s):
    import moe_expert_dispatch_amd as moe
    out = {}
    if s["case"]["kind"] == "layer":
        out["y"], residual, _ = moe.layer_norm(s["x"], s["gamma"], s["beta"], s["eps"], residual=s["residual"])
        if residual is not None:
            out["residual"] = residual
        out["dx"], out["dgamma"], out["dbeta"] = moe.layer_norm_backward(s["dy"], s["kept"], s["gamma"], s["eps"],
                                                                        dresidual=s["dresidual"])
    else:
        out["dx"], out["dgamma"] = moe.rms_norm_backward(s["dy"], s["kept"], s["gamma"], s["eps"], dresidual=s["dresidual"])
    return out


def _rows_own(s):
    import moe_expert_dispatch_amd as moe
    K = s["case"]["K"]
    out = {}
    if s["case"]["on_input"]:
        out["dy"], _ = moe.combine_backward(s["dout"], None, s["pair_row"], None, K, dy=s["dy"])
        out["dx"], out["dpair_w"] = moe.permute_backward(s["dx_perm"], s["pair_row"], K, pair_w=s["w"], x=s["x"])
    else:
        out["dy"], out["dw"] = moe.combine_backward(s["dout"], s["y"], s["pair_row"], s["w"], K, dy=s["dy"])
        out["dx"], _ = moe.permute_backward(s["dx_perm"], s["pair_row"], K)
    return out


def _experts_own(s):
    import moe_expert_dispatch_amd as moe
    off, dt = s["offsets"], s["h"].dtype
    act = moe.swiglu(s["h"], off)
    dh = moe.grouped_gemm_backward(moe.DOWN, s["dy"], off, s["w_down"], h=s["h"])
    dx = moe.grouped_gemm_backward(moe.GATE_UP_SWIGLU, dh, off, s["w_gate_up"])
    return {"act": act, "dh": dh, "dx": dx, "dw_down": moe.grouped_gemm_weight_grad(s["dy"], act, off, dw_dtype=dt),
            "dw_gate_up": moe.grouped_gemm_weight_grad(dh, s["x_perm"], off, dw_dtype=dt)}


def _weights_own(s):
    import moe_expert_dispatch_amd as moe
    return {"dw": moe.grouped_gemm_weight_grad(s["dc"], s["a"], s["offsets"], dw_dtype=torch.float32)}


def run(state):
    op = state["case"]["op"]
    if own:
        return {"norm": _norm_own, "rows": _rows_own, "experts": _experts_own, "weights": _weights_own}[op](state)
    return {"norm": _norm_plain, "rows": _rows_plain, "experts": _experts_plain, "weights": _weights_plain}[op](state)


# ---------------------------------------------------------------- least work
def work(case):
    b = _SIZE[case["dtype"]]
    if case["op"] == "norm":
        n = case["T"] * case["H"]
        res = 1 if case["residual"] else 0
        forward = 2 + 2 * res if case["kind"] == "layer" else 0
        return {"bytes": n * b * (forward + 3 + res) + case["H"] * (2 * b + 8), "flops": (20 if forward else 12) * n}
    P = case["T"] * case["K"] / case.get("ep", 1)
    if case["op"] == "rows":
        T, H, K = case["T"], case["H"], case["K"]
        if case["on_input"]:
            return {"bytes": b * H * (3 * T + 2 * P) + 16 * T * K, "flops": 4 * P * H}
        return {"bytes": b * H * (2 * T + 3 * P) + 16 * T * K, "flops": 4 * P * H}
    # experts that some token reaches, for tokens that choose K of E evenly
    E = case["E"]
    some = E * (1 - (1 - case["K"] / E) ** case["T"])
    if case["op"] == "experts":
        H, I = case["H"], case["I"]
        return {"bytes": b * (P * (3 * H + 5 * I) + 3 * H * I * (some + E)), "flops": 12 * P * H * I}
    N, Kd = case["N"], case["Kd"]
    return {"bytes": b * P * (N + Kd) + 4 * E * N * Kd, "flops": 2 * P * N * Kd}


# ---------------------------------------------------------------- 64 bits
def _norm_exact(s):
    """The definition's value, and its gradient by differentiation."""
    kind = s["case"]["kind"]
    gamma = s["gamma"].double().requires_grad_()
    beta = s["beta"].double().requires_grad_()

    def value(h):
        if kind == "rms":
            return h * torch.rsqrt((h * h).sum(1, keepdim=True) / h.shape[1] + s["eps"]) * gamma
        var, mean = torch.var_mean(h, dim=1, correction=0, keepdim=True)
        return (h - mean) / torch.sqrt(var + s["eps"]) * gamma + beta

    out = {}
    if kind == "layer":
        h = s["x"].double() + (s["residual"].double() if s["residual"] is not None else 0.0)
        with torch.no_grad():
            out["y"] = value(h)
        if s["residual"] is not None:
            out["residual"] = h
    x = s["kept"].double().requires_grad_()
    wanted = (x, gamma, beta) if kind == "layer" else (x, gamma)
    got = torch.autograd.grad(value(x), wanted, s["dy"].double())
    out["dx"] = got[0] if s["dresidual"] is None else got[0] + s["dresidual"].double()
    out["dgamma"] = got[1]
    if kind == "layer":
        out["dbeta"] = got[2]
    return out


def _rows_exact(s):
    c = s["case"]
    T, K, H = c["T"], c["K"], c["H"]
    token = s["sorted_pairs"].long() // K
    w = s["w"].double().flatten()[s["sorted_pairs"].long()]
    place = s["sorted_pairs"].long()
    out = {"dy": torch.zeros(T * K, H, dtype=torch.float64, device="cuda"),
           "dx": torch.zeros(T, H, dtype=torch.float64, device="cuda")}
    name = "dpair_w" if c["on_input"] else "dw"
    out[name] = torch.zeros(T * K, dtype=torch.float64, device="cuda")
    for at in range(0, s["rows"], 8192):  # some rows at a time
        r = slice(at, min(at + 8192, s["rows"]))
        d, back = s["dout"][token[r]].double(), s["dx_perm"][r].double()
        if c["on_input"]:
            out["dy"][r] = d
            out["dx"].index_add_(0, token[r], back * w[r, None])
            out[name][place[r]] = torch.linalg.vecdot(back, s["x"][token[r]].double())
        else:
            out["dy"][r] = d * w[r, None]
            out["dx"].index_add_(0, token[r], back)
            out[name][place[r]] = torch.linalg.vecdot(d, s["y"][r].double())
    out[name] = out[name].view(T, K)
    return out


def _experts_exact(s):
    c = s["case"]
    I, off = c["I"], s["offsets"].tolist()
    f64 = dict(dtype=torch.float64, device="cuda")
    out = {"act": torch.empty(s["rows"], I, **f64), "dh": torch.empty(s["rows"], 2 * I, **f64),
           "dx": torch.empty(s["rows"], c["H"], **f64), "dw_down": torch.zeros(s["w_down"].shape, **f64),
           "dw_gate_up": torch.zeros(s["w_gate_up"].shape, **f64)}
    for e in range(c["E"]):
        r = slice(off[e], off[e + 1])
        if off[e] == off[e + 1]:
            continue
        h = s["h"][r].double().requires_grad_()
        act = torch.nn.functional.silu(h[:, :I]) * h[:, I:]
        dy = s["dy"][r].double()
        dh, = torch.autograd.grad(act, h, torch.matmul(dy, s["w_down"][e].double()))
        act = act.detach()
        out["act"][r], out["dh"][r] = act, dh
        out["dx"][r] = torch.matmul(dh, s["w_gate_up"][e].double())
        out["dw_down"][e] = torch.matmul(dy.t(), act)
        out["dw_gate_up"][e] = torch.matmul(dh.t(), s["x_perm"][r].double())
    return out


def _weights_exact(s):
    off = s["offsets"].tolist()
    out = torch.zeros(len(off) - 1, s["dc"].shape[1], s["a"].shape[1], dtype=torch.float64, device="cuda")
    for e in range(len(off) - 1):
        out[e] = torch.matmul(s["dc"][off[e]:off[e + 1]].double().t(), s["a"][off[e]:off[e + 1]].double())
    return {"dw": out}


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _norm_exact, "rows": _rows_exact, "experts": _experts_exact, "weights": _weights_exact}[case["op"]](s)
