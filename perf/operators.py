"""Cases of the router-training operators and the dense product, and their plain forms.

Three operators:

* ``loss``: the balance loss and router z-loss of one routed batch with the per-expert counts, and the
  gradient of the logits that these two losses and the gates have together;
* ``combine_bwd``: the gradients of the gate-weighted combine: of the gates (the dot product of each token's output
  gradient with each of its selected experts' outputs), of the expert outputs, and of the zero-computation terms;
* ``linear`` / ``linear_bwd``: y = act(x W^T + b) + r and its gradients.

``own = False`` computes them with elementary torch operations in fp32, ``own = True`` by the calls a user makes.
"""

import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_LOSS_GRADS = (1e-2, 1e-3)          # upstream gradients of the two losses (their coefficients in the objective)


def listed():
    return [
        # the smallest layer's router step: launch latency
        {"name": "loss 64x8 top2", "op": "loss", "T": 64, "n_ffn": 8, "zc": False, "k": 2, "mask": False, "weight": False},
        # a MoE++ layer with zero-computation experts, a weight per expert and a padded batch
        {"name": "loss 16383x20 top2 padded", "op": "loss", "T": 16383, "n_ffn": 16, "zc": True, "k": 2, "mask": True,
         "weight": True},
        # many fine-grained experts and a large batch
        {"name": "loss 65536x256 top8", "op": "loss", "T": 65536, "n_ffn": 256, "zc": False, "k": 8, "mask": False,
         "weight": False},
        # a short MoE++ batch whose slots are partly zero, copy and constant experts
        {"name": "combine_bwd 333x2048 top2 zc", "op": "combine_bwd", "T": 333, "d": 2048, "n_ffn": 16, "zc": True, "k": 2,
         "n_shared": 0, "dtype": "bf16"},
        # a large long-tail batch, six routed and two shared experts per token
        {"name": "combine_bwd 8192x2048 top6", "op": "combine_bwd", "T": 8192, "d": 2048, "n_ffn": 64, "zc": False, "k": 6,
         "n_shared": 2, "dtype": "bf16"},
        # one generated token through a square projection: the weights are read once
        {"name": "linear 1x4096x4096", "op": "linear", "M": 1, "N": 4096, "K": 4096, "dtype": "bf16", "act": "none",
         "out_f32": False, "bias": True, "residual": True, "save": False, "pad": 0},
        # router logits with the gating residual of the previous layer
        {"name": "linear router 16384x20x2048", "op": "linear", "M": 16384, "N": 20, "K": 2048, "dtype": "bf16",
         "act": "none", "out_f32": True, "bias": True, "residual": True, "save": False, "pad": 0},
        # odd sizes everywhere, the pre-activation kept for the backward pass
        {"name": "linear odd 333x1029x1411", "op": "linear", "M": 333, "N": 1029, "K": 1411, "dtype": "bf16", "act": "gelu",
         "out_f32": False, "bias": True, "residual": True, "save": True, "pad": 0},
        # the first product of a dense feed-forward block
        {"name": "linear 8192x14336x4096", "op": "linear", "M": 8192, "N": 14336, "K": 4096, "dtype": "bf16", "act": "gelu",
         "out_f32": False, "bias": True, "residual": False, "save": False, "pad": 0},
        # the router's weights and input gradients from fp32 logit gradients
        {"name": "linear_bwd router 16384x20x2048", "op": "linear_bwd", "M": 16384, "N": 20, "K": 2048, "dtype": "bf16",
         "act": "none", "out_f32": True, "grad_f32": True, "bias": True, "pad": 0},
        # a dense projection's training step
        {"name": "linear_bwd 8192x4096x4096", "op": "linear_bwd", "M": 8192, "N": 4096, "K": 4096, "dtype": "bf16",
         "act": "silu", "out_f32": False, "grad_f32": False, "bias": True, "pad": 0},
        # the small fp32 layer's sizes, odd in every direction
        {"name": "linear_bwd f32 201x77x129", "op": "linear_bwd", "M": 201, "N": 77, "K": 129, "dtype": "f32", "act": "gelu",
         "out_f32": False, "grad_f32": False, "bias": True, "pad": 3},
    ]


_MOST_FLOPS = 2 * 8192 * 14336 * 4096


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["loss", "combine_bwd", "linear", "linear", "linear_bwd", "linear_bwd"])
    if op == "loss":
        n = _log(rng, 2, 252)
        return {"op": op, "T": _log(rng, 1, 60000), "n_ffn": n, "zc": rng.random() < 0.4, "k": _log(rng, 1, min(n, 16)),
                "mask": rng.random() < 0.5, "weight": rng.random() < 0.5}
    if op == "combine_bwd":
        n = _log(rng, 2, 128)
        k, d, ns = _log(rng, 1, min(n, 8)), 64 * _log(rng, 1, 64), rng.choice([0, 0, 1, 2])
        T = min(_log(rng, 1, 16384), 8192 * 2048 * 4 // ((k + ns) * d))
        return {"op": op, "T": T, "d": d, "n_ffn": n, "zc": rng.random() < 0.5, "k": k, "n_shared": ns,
                "dtype": "f32" if rng.random() < 0.2 else "bf16"}
    f32 = rng.random() < 0.2
    N = _log(rng, 1, 2048 if f32 else 14336)
    K = _log(rng, 8, 2048 if f32 else 8192)
    M = _log(rng, 1, 4096 if f32 else 16384)
    if rng.random() < 0.5:      # widths that a model has
        N, K = 8 * ((N + 7) // 8), 64 * ((K + 63) // 64)
    M = max(1, min(M, _MOST_FLOPS // ((2 if op == "linear" else 6) * N * K)))
    act = rng.choice(["none", "relu", "silu", "gelu"])
    case = {"op": op, "M": M, "N": N, "K": K, "dtype": "f32" if f32 else "bf16", "act": act, "out_f32": rng.random() < 0.3,
            "bias": rng.random() < 0.7, "pad": rng.choice([0, 0, 8, 24, 5])}
    if op == "linear":
        case.update(residual=rng.random() < 0.5, save=act != "none" and rng.random() < 0.5)
    else:
        case.update(grad_f32=rng.random() < 0.3)
    return case


def _widths(case):
    zc = (1, 1, 2) if case["zc"] else (0, 0, 0)
    return case["n_ffn"], zc, case["n_ffn"] + sum(zc)


def _layer_desc(case, d, dtype):
    import mixture_experts_layer_swiglu_b200 as moe
    n_ffn, (n_zero, n_copy, n_const), _ = _widths(case)
    n_shared = case.get("n_shared", 0)
    return moe.make_desc(T=case["T"], d_model=d, top_k=case["k"], dtype=dtype, n_ffn=n_ffn, hidden=128, n_zero=n_zero,
                         n_copy=n_copy, n_const=n_const, n_shared=n_shared, hidden_shared=128 if n_shared else 0)


def _linear_desc(case):
    import mixture_experts_layer_swiglu_b200 as moe
    return moe.make_linear_desc(M=case["M"], N=case["N"], K=case["K"], dtype=case["dtype"], act=case["act"],
                                out_f32=case["out_f32"], grad_f32=case.get("grad_f32", False),
                                ld_x=case["K"] + case["pad"])


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, std=1.0, dtype=torch.float32):
        return (torch.randn(shape, device="cuda", generator=g) * std).to(dtype)

    s = {"case": case}
    if case["op"] == "loss":
        T, k = case["T"], case["k"]
        _, _, E = _widths(case)
        # trained routers prefer some experts: a fixed offset per expert on top of the tokens' own logits
        s["logits"] = normal(T, E, std=1.5) + normal(E, std=0.7)
        top, idx = torch.sort(s["logits"], dim=1, descending=True, stable=True)
        s["idx"] = idx[:, :k].to(torch.int32).contiguous()
        s["gate"] = torch.softmax(top[:, :k], dim=1).contiguous()
        s["dgate"] = normal(T, k, std=1.0 / T)
        s["mask"] = (torch.arange(T, device="cuda") % 512 < 448).to(torch.uint8) if case["mask"] else None
        s["weight"] = torch.where(torch.arange(E, device="cuda") < case["n_ffn"], 1.0, 0.5) if case["weight"] else None
        s["dlosses"] = torch.tensor(_LOSS_GRADS, device="cuda")
        if own:
            import mixture_experts_layer_swiglu_b200 as moe
            s["desc"] = _layer_desc(case, 64, "bf16")
            s["bufs"] = moe.RouterGradBuffers(s["desc"])
        return s
    if case["op"] == "combine_bwd":
        T, d, k, dt, n_shared = case["T"], case["d"], case["k"], _DT[case["dtype"]], case["n_shared"]
        n_ffn, (_, _, n_const), E = _widths(case)
        s["idx"] = torch.rand((T, E), device="cuda", generator=g).argsort(dim=1)[:, :k].to(torch.int32).contiguous()
        s["gate"] = torch.softmax(normal(T, k), dim=1)
        # rows in (expert, token) order; the shared experts' rows follow the routed ones
        flat = s["idx"].reshape(-1)
        order = torch.argsort(flat, stable=True)
        row = torch.empty_like(order)
        row[order] = torch.arange(T * k, device="cuda")
        s["row_of"] = torch.where(flat < n_ffn, row, -1).to(torch.int32).reshape(T, k).contiguous()
        ends = torch.searchsorted(flat[order].contiguous(), torch.arange(n_ffn + 1, device="cuda", dtype=torch.int32))
        shared = ends[-1] + T * torch.arange(1, n_shared + 1, device="cuda")
        s["offsets"] = torch.cat([ends, shared]).to(torch.int32)
        s["y_sorted"] = normal(T * (k + n_shared), d)
        s["dy"], s["x"] = normal(T, d, dtype=dt), normal(T, d, dtype=dt)
        s["const_vec"] = normal(n_const, d, dtype=dt)
        s["const_mix"] = torch.softmax(normal(T, n_const, 2), dim=-1)
        s["dgate"] = torch.empty((T, k), device="cuda")
        # rows past the last group belong to no slot: they keep what they hold
        s["dy_sorted"] = torch.zeros((T * (k + n_shared), d), dtype=dt, device="cuda")
        s["dx"] = torch.empty((T, d), dtype=dt, device="cuda")
        s["dconst_mix"] = torch.empty((T, n_const, 2), device="cuda")
        s["dconst_vec"] = torch.empty((n_const, d), device="cuda")
        if own:
            s["desc"] = _layer_desc(case, d, case["dtype"])
        return s
    M, N, K, dt = case["M"], case["N"], case["K"], _DT[case["dtype"]]
    out = torch.float32 if case["out_f32"] else dt
    s["x"] = normal(M, K + case["pad"], dtype=dt)[:, :K]
    s["w"] = normal(N, K, std=K ** -0.5, dtype=dt)
    s["bias"] = normal(N, std=0.5) if case["bias"] else None
    if case["op"] == "linear":
        s["residual"] = normal(M, N, dtype=out) if case["residual"] else None
    else:
        s["dy"] = normal(M, N, dtype=out)
        s["z"] = normal(M, N, dtype=dt) if case["act"] != "none" else None
    if own:
        import mixture_experts_layer_swiglu_b200 as moe
        s["layer"] = moe.Linear(_linear_desc(case), s["w"], s["bias"])
    return s


# ------------------------------------------------------------ plain forms

def _plain_loss(s):
    z, k = s["logits"], s["case"]["k"]
    T, E = z.shape
    idx = s["idx"].long()
    m = s["mask"].to(torch.int32) if s["mask"] is not None else torch.ones(T, dtype=torch.int32, device=z.device)
    counts = torch.zeros(E + 1, dtype=torch.int32, device=z.device)
    counts.scatter_add_(0, idx.reshape(-1), m.repeat_interleave(k))
    n = m.sum()
    counts[E] = n
    top = z.amax(dim=1, keepdim=True)
    e = torch.exp(z - top)
    total = e.sum(dim=1, keepdim=True)
    p = e / total
    lse = top + torch.log(total)
    mf = m.float()[:, None]
    inv = torch.where(n > 0, 1.0 / n.float(), 0.0)
    prob_mean = (p * mf).sum(dim=0) * inv
    f = counts[:E].float() * inv / k
    wf = f * s["weight"] if s["weight"] is not None else f
    losses = torch.stack([E * (wf * prob_mean).sum(), (lse * lse * mf).sum() * inv])
    db, dz = s["dlosses"][0], s["dlosses"][1]
    grad = mf * inv * p * (db * E * (wf - (p * wf).sum(dim=1, keepdim=True)) + 2 * dz * lse)
    gg = s["gate"] * (s["dgate"] - (s["gate"] * s["dgate"]).sum(dim=1, keepdim=True))
    return {"losses": losses, "prob_mean": prob_mean, "counts": counts, "dlogits": grad.scatter_add(1, idx, gg)}


def _plain_combine_bwd(s):
    case, dt = s["case"], s["x"].dtype
    T, k, n_shared = case["T"], case["k"], case["n_shared"]
    n_ffn, (n_zero, n_copy, n_const), _ = _widths(case)
    dy, x, gate = s["dy"].float(), s["x"].float(), s["gate"]
    idx, row = s["idx"].long(), s["row_of"].long()
    dgate = (s["y_sorted"][row.clamp(min=0)] * dy[:, None]).sum(dim=-1)
    # one row more than the buffer takes the slots that have none; shared rows start where the groups say
    rows = s["dy_sorted"].shape[0]
    dys = torch.zeros((rows + 1, case["d"]), device=dy.device)
    dys[torch.where(row < 0, rows, row)] = gate[:, :, None] * dy[:, None]
    if n_shared:
        at = s["offsets"][n_ffn:n_ffn + n_shared].long()[:, None] + torch.arange(T, device=dy.device)
        dys[at] = dy.expand(n_shared, T, case["d"])
    out = {"dy_sorted": dys[:rows].to(dt)}
    if not case["zc"]:
        return {"dgate": dgate, **out}
    first = n_ffn + n_zero + n_copy
    is_copy, is_const = (idx >= n_ffn + n_zero) & (idx < first), idx >= first
    copy = (x * dy).sum(dim=-1, keepdim=True)
    vec = dy @ s["const_vec"].float().T
    hit = is_const[:, :, None] & (idx[:, :, None] - first == torch.arange(n_const, device=dy.device))
    weight = (gate[:, :, None] * hit).sum(dim=1)                     # [T, n_const]: the slots' gates of each constant expert
    a1, a2 = s["const_mix"][:, :, 0], s["const_mix"][:, :, 1]
    const = ((a1 * copy + a2 * vec)[:, None] * hit).sum(dim=-1)
    out["dgate"] = torch.where(is_const, const, torch.where(is_copy, copy, torch.where(idx < n_ffn, dgate, 0.0)))
    out["dx"] = (((gate * is_copy).sum(dim=1, keepdim=True) + (weight * a1).sum(dim=1, keepdim=True)) * dy).to(dt)
    out["dconst_mix"] = torch.stack([weight * copy, weight * vec], dim=-1)
    out["dconst_vec"] = (weight * a2).T @ dy
    return out


def _act(z, act):
    if act == "relu":
        return z * (z > 0)
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    return z


def _act_grad(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "silu":
        sg = 1 / (1 + torch.exp(-z))
        return sg * (1 + z * (1 - sg))
    return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)


def _plain_linear(s):
    case, dt = s["case"], s["x"].dtype
    out = torch.float32 if case["out_f32"] else dt
    z = s["x"].float() @ s["w"].float().T
    if s["bias"] is not None:
        z = z + s["bias"]
    y = _act(z, case["act"])
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return {"y": y.to(out), "z": z.to(dt)} if case["save"] else {"y": y.to(out)}


def _plain_linear_bwd(s):
    case, dt = s["case"], s["x"].dtype
    dz = s["dy"].float()
    if case["act"] != "none":
        dz = dz * _act_grad(s["z"].float(), case["act"])
    dw = dz.T @ s["x"].float()
    return {"dx": (dz @ s["w"].float()).to(dt), "dw": dw if case["grad_f32"] else dw.to(dt),
            "db": dz.sum(dim=0) if case["bias"] else None}


def run(state):
    case = state["case"]
    op = case["op"]
    if not own:
        return {"loss": _plain_loss, "combine_bwd": _plain_combine_bwd, "linear": _plain_linear, "linear_bwd": _plain_linear_bwd}[op](state)
    import mixture_experts_layer_swiglu_b200 as moe
    if op == "loss":
        b = state["bufs"]
        moe.moe_balance_loss(state["desc"], state["logits"], state["idx"], state["mask"], state["weight"], b.counts,
                             b.prob_mean, b.losses, b.workspace)
        moe.moe_route_backward(state["desc"], state["logits"], state["idx"], state["gate"], state["dgate"], state["mask"],
                               state["weight"], b.counts, state["dlosses"], b.dlogits)
        return {"losses": b.losses, "prob_mean": b.prob_mean, "counts": b.counts, "dlogits": b.dlogits}
    if op == "combine_bwd":
        zc = case["zc"]
        moe.moe_combine_backward(state["desc"], {"const_vec": state["const_vec"]} if zc else {}, state["dy"],
                                 state["y_sorted"], state["offsets"], state["row_of"], state["idx"], state["gate"],
                                 state["const_mix"] if zc else None, state["x"] if zc else None, state["dgate"],
                                 state["dy_sorted"], state["dx"] if zc else None, state["dconst_mix"] if zc else None,
                                 state["dconst_vec"] if zc else None)
        return {n: state[n] for n in ("dgate", "dy_sorted") + (("dx", "dconst_mix", "dconst_vec") if zc else ())}
    if op == "linear":
        z = torch.empty((case["M"], case["N"]), dtype=state["x"].dtype, device="cuda") if case["save"] else None
        y = state["layer"].forward(state["x"], residual=state["residual"], z=z)
        return {"y": y, "z": z} if case["save"] else {"y": y}
    dx, dw, db = state["layer"].backward(state["x"], state["dy"], z=state["z"])
    return {"dx": dx, "dw": dw, "db": db}


def work(case):
    if case["op"] == "loss":
        T, k = case["T"], case["k"]
        _, _, E = _widths(case)
        # logits in, their gradient out, indices, gates and gate gradients in; exp, sums and the two products per logit
        return {"bytes": T * (8 * E + 12 * k + (1 if case["mask"] else 0)) + 12 * E, "flops": 14 * T * E}
    if case["op"] == "combine_bwd":
        T, d, k, n_shared = case["T"], case["d"], case["k"], case["n_shared"]
        n_ffn, (_, _, n_const), E = _widths(case)
        el = 4 if case["dtype"] == "f32" else 2
        rows = T * k * n_ffn / E
        zc = 2 * T * d * el + 2 * T * n_const * 8 + n_const * d * (4 + el) if case["zc"] else 0
        return {"bytes": int(rows * d * (4 + el) + n_shared * T * d * el + T * d * el + T * k * 16 + zc),
                "flops": int(3 * rows * d + (8 * T * d if case["zc"] else 0))}
    M, N, K = case["M"], case["N"], case["K"]
    el = 4 if case["dtype"] == "f32" else 2
    out = 4 if case["out_f32"] else el
    if case["op"] == "linear":
        return {"bytes": el * (M * K + N * K) + out * M * N * (2 if case["residual"] else 1) + (4 * N if case["bias"] else 0)
                + (el * M * N if case["save"] else 0), "flops": 2 * M * N * K}
    z = el * M * N if case["act"] != "none" else 0
    return {"bytes": 2 * el * M * K + N * K * (el + (4 if case["grad_f32"] else el)) + out * M * N + z
            + (4 * N if case["bias"] else 0), "flops": 4 * M * N * K}


# ------------------------------------------------------------ the definitions in 64 bits

def _exact_loss(s):
    z, idx, k = s["logits"].double(), s["idx"].long(), s["case"]["k"]
    T, E = z.shape
    live = s["mask"].bool() if s["mask"] is not None else torch.ones(T, dtype=torch.bool, device=z.device)
    n = int(live.sum())
    chosen = torch.zeros_like(z).scatter_(1, idx, 1.0)
    counts = chosen[live].sum(dim=0)
    lse = torch.logsumexp(z, dim=1)
    p = torch.exp(z - lse[:, None])
    w = s["weight"].double() if s["weight"] is not None else torch.ones(E, dtype=torch.float64, device=z.device)
    load = w * counts / max(n * k, 1)
    prob_mean = p[live].sum(dim=0) / max(n, 1)
    losses = torch.stack([E * torch.dot(load, prob_mean), lse[live].square().sum() / max(n, 1)])
    cb, cz = (float(v) for v in s["dlosses"])
    d = cb * E * p * (load[None, :] - (p @ load)[:, None]) + 2 * cz * lse[:, None] * p
    d = torch.where(live[:, None], d / max(n, 1), 0.0)
    gate, dgate = s["gate"].double(), s["dgate"].double()
    mean = torch.einsum("tk,tk->t", gate, dgate)
    d.scatter_add_(1, idx, gate * (dgate - mean[:, None]))
    return {"losses": losses, "prob_mean": prob_mean,
            "counts": torch.cat([counts, counts.new_tensor([n])]).to(torch.int32), "dlogits": d}


def _exact_combine_bwd(s):
    case = s["case"]
    n_ffn, (n_zero, n_copy, n_const), _ = _widths(case)
    T, k = s["idx"].shape
    dy, x, gate = s["dy"].double(), s["x"].double(), s["gate"].double()
    f64 = dict(dtype=torch.float64, device=dy.device)
    dgate, dys = torch.zeros((T, k), **f64), torch.zeros(s["dy_sorted"].shape, **f64)
    dx, dmix, dvec = torch.zeros_like(x), torch.zeros(s["dconst_mix"].shape, **f64), torch.zeros((n_const, case["d"]), **f64)
    for i in range(case["n_shared"]):
        lo = int(s["offsets"][n_ffn + i])
        dys[lo:lo + T] = dy
    for j in range(k):
        e, r = s["idx"][:, j].long(), s["row_of"][:, j].long()
        at = torch.nonzero(e < n_ffn).reshape(-1)
        dgate[at, j] = torch.einsum("td,td->t", s["y_sorted"][r[at]].double(), dy[at])
        dys[r[at]] = gate[at, j, None] * dy[at]
        at = torch.nonzero((e >= n_ffn + n_zero) & (e < n_ffn + n_zero + n_copy)).reshape(-1)
        dgate[at, j] = torch.einsum("td,td->t", x[at], dy[at])
        dx[at] += gate[at, j, None] * dy[at]
        for c in range(n_const):
            at = torch.nonzero(e == n_ffn + n_zero + n_copy + c).reshape(-1)
            a, v, g = s["const_mix"][at, c].double(), s["const_vec"][c].double(), gate[at, j]
            along, onto = torch.einsum("td,td->t", x[at], dy[at]), torch.einsum("d,td->t", v, dy[at])
            dgate[at, j] = a[:, 0] * along + a[:, 1] * onto
            dx[at] += (g * a[:, 0])[:, None] * dy[at]
            dmix[at, c] = torch.stack([g * along, g * onto], dim=1)
            dvec[c] += torch.einsum("t,td->d", g * a[:, 1], dy[at])
    out = {"dgate": dgate, "dy_sorted": dys}
    return {**out, "dx": dx, "dconst_mix": dmix, "dconst_vec": dvec} if case["zc"] else out


def _phi(z):
    return 0.5 * torch.special.erfc(-z / math.sqrt(2.0))


def _exact_linear(s):
    z = torch.einsum("mk,nk->mn", s["x"].double(), s["w"].double())
    if s["bias"] is not None:
        z += s["bias"].double()
    act = s["case"]["act"]
    y = {"none": lambda: z, "relu": lambda: z.clamp(min=0), "silu": lambda: z * torch.sigmoid(z),
         "gelu": lambda: z * _phi(z)}[act]()
    if s["residual"] is not None:
        y = y + s["residual"].double()
    return {"y": y, "z": z} if s["case"]["save"] else {"y": y}


def _exact_linear_bwd(s):
    dz, act = s["dy"].double(), s["case"]["act"]
    if act != "none":
        z = s["z"].double()
        slope = {"relu": lambda: (z > 0).double(),
                 "silu": lambda: torch.sigmoid(z) + z * torch.sigmoid(z) * torch.sigmoid(-z),
                 "gelu": lambda: _phi(z) + z * torch.exp(-z.square() / 2) * (2 * math.pi) ** -0.5}[act]()
        dz = dz * slope
    return {"dx": torch.einsum("mn,nk->mk", dz, s["w"].double()), "dw": torch.einsum("mn,mk->nk", dz, s["x"].double()),
            "db": dz.sum(dim=0) if s["case"]["bias"] else None}


def exact(case, seed):
    s = prepare(case, seed)
    return {"loss": _exact_loss, "combine_bwd": _exact_combine_bwd, "linear": _exact_linear, "linear_bwd": _exact_linear_bwd}[case["op"]](s)
