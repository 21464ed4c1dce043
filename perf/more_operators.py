"""Rows between token order and expert order, and the dense product beside the experts, as measured cases.

Each case is one pass; `op` names it:

* dispatch     tokens' rows to expert order, and the gradient of that (a token's rows summed)
* combine      a token's expert rows summed with their routing weights onto the residual, and, in training, its gradient
* linear       act(x W^T + b) + residual
* linear_grad  gradients of a layer's input (through the activation that made it), weight and bias
* act_grad     the gradient through an activation that is a layer's last step

`own` selects the framework's kernels; otherwise `run` computes the plain form in elementary torch operations.
"""
import math

import torch

own = False

DEV = "cuda"
ACTS = ("none", "relu", "silu", "gelu_tanh")


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # a few short sequences on their way to the experts; a training batch of long ones, with pairs that no expert takes
        {"name": "dispatch short batch", "op": "dispatch", "T": 203, "k": 8, "E": 128, "H": 2048, "drop": False},
        {"name": "dispatch training batch", "op": "dispatch", "T": 16384, "k": 8, "E": 256, "H": 6144, "drop": True},
        # the experts' rows of one decoded token; a training batch, forward and backward
        {"name": "combine decode one token", "op": "combine", "T": 1, "k": 8, "E": 256, "H": 6144, "drop": False, "residual": True, "grad": False},
        {"name": "combine training batch", "op": "combine", "T": 16384, "k": 8, "E": 256, "H": 6144, "drop": True, "residual": True, "grad": True},
        # a shared expert's gate/up product for one decoded token; its down product for a small serving batch
        {"name": "linear decode one token", "op": "linear", "M": 1, "N": 4096, "K": 6144, "act": "none", "bias": False, "residual": False, "keep": False},
        {"name": "linear serving batch", "op": "linear", "M": 37, "N": 6144, "K": 2048, "act": "none", "bias": False, "residual": True, "keep": False},
        # a short prefill through a dense layer, sizes that are no multiple of a tile
        {"name": "linear ragged prefill", "op": "linear", "M": 1111, "N": 2848, "K": 2080, "act": "gelu_tanh", "bias": True, "residual": True, "keep": False},
        # a training batch; the pre-activation is kept for the backward
        {"name": "linear training batch", "op": "linear", "M": 16384, "N": 4096, "K": 6144, "act": "silu", "bias": True, "residual": False, "keep": True},
        # fine-tuning on a few short sequences; a training batch
        {"name": "linear_grad short batch", "op": "linear_grad", "M": 203, "N": 2048, "K": 768, "act": "gelu_tanh", "add": False},
        {"name": "linear_grad training batch", "op": "linear_grad", "M": 16384, "N": 4096, "K": 6144, "act": "silu", "add": True},
        # a layer that ends with its activation: a few short sequences; a training batch
        {"name": "act_grad short batch", "op": "act_grad", "M": 203, "N": 768, "act": "silu"},
        {"name": "act_grad training batch", "op": "act_grad", "M": 16384, "N": 4096, "act": "gelu_tanh"},
    ]


def _between(rng, lo, hi, step=1):
    """A multiple of step in [lo, hi], spread evenly over the logarithm."""
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi)))) // step * step))


def draw(rng):
    op = rng.choice(("dispatch", "combine", "combine", "linear", "linear", "linear_grad", "linear_grad", "act_grad"))
    if op in ("dispatch", "combine"):
        k = rng.choice((1, 2, 4, 6, 8))
        c = {"op": op, "T": _between(rng, 1, 16384), "k": k, "E": rng.choice((8, 16, 60, 64, 128, 256)), "H": _between(rng, 64, 6144, 8), "drop": rng.random() < 0.5}
        return c if op == "dispatch" else {**c, "residual": rng.random() < 0.5, "grad": rng.random() < 0.6}
    if op == "act_grad":
        return {"op": op, "M": _between(rng, 1, 16384), "N": _between(rng, 64, 4096, 8), "act": rng.choice(ACTS[1:])}
    M, N, K = _between(rng, 1 if op == "linear" else 16, 8192), _between(rng, 64, 8192, 8), _between(rng, 64, 8192, 8)
    while M * N * K > 1 << 38:  # a drawn case stays under the largest listed one
        N, K = max(64, N // 16 * 8), max(64, K // 16 * 8)
    c = {"op": op, "M": M, "N": N, "K": K, "act": rng.choice(ACTS)}
    if op == "linear":
        return {**c, "bias": rng.random() < 0.5, "residual": rng.random() < 0.5, "keep": rng.random() < 0.3}
    return {**c, "add": rng.random() < 0.5}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _normal(g, shape, std=1.0):
    return torch.randn(shape, generator=g, device=DEV).mul_(std).to(torch.bfloat16)


def _routing(g, T, E, k, drop):
    """Places of the routed pairs in expert order, as the framework's permutation gives them, and how many have an expert."""
    score = torch.rand((T, E), generator=g, device=DEV)
    idx = score.topk(k, dim=1).indices.flatten()
    if drop:  # pairs that are switched off stand behind every expert's
        idx = torch.where(torch.rand(T * k, generator=g, device=DEV) < 0.05, E, idx)
    perm = torch.argsort(idx, stable=True)
    inv = torch.empty_like(perm).scatter_(0, perm, torch.arange(T * k, device=DEV))
    return inv.int(), (idx < E).sum().int().reshape(1)


def _activation(v, act):
    """act(v), and act'(v)."""
    if act == "none":
        return v, torch.ones_like(v)
    if act == "relu":
        return torch.where(v > 0, v, 0.0), (v > 0).to(v.dtype)
    if act == "silu":
        s = 1 / (1 + torch.exp(-v))
        return v * s, s * (1 + v * (1 - s))
    c = 2 * math.sqrt(2 / math.pi)
    s = 1 / (1 + torch.exp(-c * (v + 0.044715 * v * v * v)))  # (1 + tanh(u)) / 2 with 2 u in place of u
    return v * s, s + v * s * (1 - s) * c * (1 + 3 * 0.044715 * v * v)


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device=DEV).manual_seed(int(seed) * 1_000_003 + 29)
    op = c["op"]
    empty = lambda *shape, dtype=torch.bfloat16: torch.empty(shape, dtype=dtype, device=DEV)  # noqa: E731
    if op in ("dispatch", "combine"):
        T, k, H = c["T"], c["k"], c["H"]
        inv, n = _routing(g, T, c["E"], k, c["drop"])
        rows = _normal(g, (T * k, H))
        if c["drop"]:  # rows of pairs that no expert took hold whatever was there
            rows[torch.arange(T * k, device=DEV) >= n] = float("nan")
        s = {**c, "inv": inv, "n": n, "x": _normal(g, (T, H)), "rows": rows, "out": torch.zeros_like(rows), "y": empty(T, H)}
        s["w"] = torch.rand((T, k), generator=g, device=DEV)
        s["dw"] = empty(T, k, dtype=torch.float32)
        s["dout"] = _normal(g, (T, H))
        return s
    if op == "act_grad":
        shape = (c["M"], c["N"])
        return {**c, "dy": _normal(g, shape), "z": _normal(g, shape, 1.5), "dz": empty(*shape)}
    M, N, K = c["M"], c["N"], c["K"]
    s = {**c, "w": _normal(g, (N, K), 1 / math.sqrt(K)), "ws": None}
    if op == "linear":
        s.update(x=_normal(g, (M, K)), b=_normal(g, (N,), 0.5) if c["bias"] else None, r=_normal(g, (M, N)) if c["residual"] else None,
                 y=empty(M, N), z=empty(M, N) if c["keep"] else None)
    else:
        s.update(zx=_normal(g, (M, K), 1.5), dz=_normal(g, (M, N)), add=_normal(g, (M, K)) if c["add"] else None, dx=empty(M, K),
                 dw=empty(N, K, dtype=torch.float32), db=empty(N, dtype=torch.float32))
        s["x"] = torch.empty_like(s["zx"])
        for i in range(0, M, 4096):
            s["x"][i:i + 4096] = _activation(s["zx"][i:i + 4096].float(), c["act"])[0].to(torch.bfloat16)
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _plain_sum(rows, inv, n, w, k):
    """Each token's rows, weighted and summed; those of pairs without an expert count as nothing."""
    at = inv.long()
    kept = at < n
    v = rows[torch.where(kept, at, 0)].float()
    v = torch.where(kept.unsqueeze(-1), v, 0.0).unflatten(0, (-1, k))
    return v.sum(1) if w is None else (v * w.unsqueeze(-1)).sum(1)


def _plain_dispatch(s):
    at = s["inv"].long()
    kept = torch.nonzero(at < s["n"]).flatten()
    out = torch.zeros_like(s["rows"])
    out[at[kept]] = s["x"][kept // s["k"]]
    return {"rows": out, "dx": _plain_sum(s["rows"], s["inv"], s["n"], None, s["k"]).to(torch.bfloat16)}


def _plain_combine(s):
    k = s["k"]
    y = _plain_sum(s["rows"], s["inv"], s["n"], s["w"], k)
    out = {"y": (y + s["x"].float() if s["residual"] else y).to(torch.bfloat16)}
    if s["grad"]:
        at = s["inv"].long()
        kept = at < s["n"]
        pairs = torch.nonzero(kept).flatten()
        d = s["dout"].float()
        dy = torch.zeros_like(s["rows"])
        dy[at[pairs]] = (d[pairs // k] * s["w"].flatten()[pairs].unsqueeze(-1)).to(torch.bfloat16)
        v = torch.where(kept.unsqueeze(-1), s["rows"][at].float(), 0.0).unflatten(0, (-1, k))
        out.update(dy=dy, dw=(v * d.unsqueeze(1)).sum(-1))
    return out


def _plain_linear(s):
    z = s["x"].float() @ s["w"].float().T
    if s["b"] is not None:
        z = z + s["b"].float()
    y = _activation(z, s["act"])[0]
    if s["r"] is not None:
        y = y + s["r"].float()
    out = {"y": y.to(torch.bfloat16)}
    if s["keep"]:
        out["z"] = z.to(torch.bfloat16)
    return out


def _plain_linear_grad(s):
    dz = s["dz"].float()
    dx = dz @ s["w"].float()
    if s["act"] != "none":
        dx = dx * _activation(s["zx"].float(), s["act"])[1]
    if s["add"] is not None:
        dx = dx + s["add"].float()
    return {"dx": dx.to(torch.bfloat16), "dw": dz.T @ s["x"].float(), "db": dz.sum(0)}


def _plain_act_grad(s):
    return (s["dy"].float() * _activation(s["z"].float(), s["act"])[1]).to(torch.bfloat16)


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def _workspace(bqm, s):
    """The product's scratch memory, made by the first pass and kept, as a user's program keeps it."""
    if s["ws"] is None:
        s["ws"] = torch.empty(max(16, bqm.bqm_linear_workspace_size(s["M"], s["N"], s["K"])), dtype=torch.uint8, device=DEV)
    return s["ws"]


def _own(s):
    import bit_quantized_moe_amd as bqm
    op = s["op"]
    if op == "dispatch":
        bqm.bqm_dispatch(s["x"], s["inv"], s["out"], n_rows=s["n"])
        return {"rows": s["out"], "dx": bqm.bqm_combine(s["rows"], s["inv"], s["y"], n_rows=s["n"])}
    if op == "combine":
        out = {"y": bqm.bqm_combine(s["rows"], s["inv"], s["y"], topk_w=s["w"], residual=s["x"] if s["residual"] else None, n_rows=s["n"])}
        if s["grad"]:
            bqm.bqm_combine_grad(s["dout"], s["inv"], y=s["rows"], topk_w=s["w"], dy=s["out"], dtopk_w=s["dw"], n_rows=s["n"])
            out.update(dy=s["out"], dw=s["dw"])
        return out
    act = getattr(bqm, "ACT_" + s["act"].upper())
    if op == "act_grad":
        return bqm.bqm_act_grad(s["dy"], s["z"], act, s["dz"])
    ws = _workspace(bqm, s)
    if op == "linear":
        bqm.bqm_linear_fwd(s["x"], s["w"], s["y"], bias=s["b"], act=act, residual=s["r"], z=s["z"], ws=ws)
        return {"y": s["y"], "z": s["z"]} if s["keep"] else {"y": s["y"]}
    bqm.bqm_linear_dgrad(s["dz"], s["w"], s["dx"], zx=None if s["act"] == "none" else s["zx"], act=act, add=s["add"], ws=ws)
    bqm.bqm_linear_wgrad(s["dz"], s["x"], s["dw"], dbias=s["db"], ws=ws)
    return {"dx": s["dx"], "dw": s["dw"], "db": s["db"]}


def run(state):
    if own:
        return _own(state)
    return {"dispatch": _plain_dispatch, "combine": _plain_combine, "linear": _plain_linear, "linear_grad": _plain_linear_grad,
            "act_grad": _plain_act_grad}[state["op"]](state)


def work(case):
    c = case
    op = c["op"]
    if op in ("dispatch", "combine"):
        t, r = c["T"] * c["H"] * 2, c["T"] * c["k"] * c["H"] * 2  # bytes of the tokens' rows and of the experts'
        small = 4 * c["T"] * c["k"]
        if op == "dispatch":  # x to rows, rows to dx
            return {"bytes": 2 * (t + r + small), "flops": r // 2}
        moved = r + t * (2 if c["residual"] else 1) + 2 * small
        if c["grad"]:  # dout and the rows read, dy and dw written
            moved += t + 2 * r + 3 * small
        return {"bytes": moved, "flops": r * (2 if c["grad"] else 1)}
    if op == "act_grad":
        n = c["M"] * c["N"]
        return {"bytes": 6 * n, "flops": 10 * n}
    M, N, K = c["M"], c["N"], c["K"]
    if op == "linear":
        return {"bytes": 2 * (M * K + N * K + M * N * (1 + c["residual"] + c["keep"]) + N * c["bias"]), "flops": 2 * M * N * K}
    return {"bytes": 2 * (M * N + N * K + M * K * (2 + (c["act"] != "none") + c["add"])) + 4 * (N * K + N), "flops": 4 * M * N * K}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _exact_act(v, act, order):
    """act(v) (order 0) or act'(v) (order 1) of float64 values."""
    if act == "none":
        return v if order == 0 else torch.ones_like(v)
    if act == "relu":
        return v.clamp(min=0) if order == 0 else torch.heaviside(v, torch.zeros_like(v))
    if act == "silu":
        s = torch.sigmoid(v)
        return v * s if order == 0 else s + v * s * (1 - s)
    t = torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3))
    if order == 0:
        return 0.5 * v * (1 + t)
    return 0.5 * (1 + t) + 0.5 * v * (1 - t ** 2) * math.sqrt(2 / math.pi) * (1 + 0.134145 * v ** 2)


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op in ("dispatch", "combine"):
        T, k, H, n = s["T"], s["k"], s["H"], int(s["n"])
        inv = s["inv"].long().view(T, k)
        total = torch.zeros((T, H), dtype=torch.float64, device=DEV)
        moved = torch.zeros((T * k, H), dtype=torch.float64, device=DEV)
        dots = torch.zeros((T, k), dtype=torch.float64, device=DEV)
        for j in range(k):
            t = torch.nonzero(inv[:, j] < n).flatten()
            at = inv[t, j]
            w = s["w"][t, j].double().unsqueeze(1) if op == "combine" else 1.0
            rows = s["rows"][at].double()
            total[t] += rows * w
            if op == "dispatch":
                moved[at] = s["x"][t].double()
            elif s["grad"]:
                d = s["dout"][t].double()
                moved[at] = d * w
                dots[t, j] = torch.linalg.vecdot(d, rows)
        if op == "dispatch":
            return {"rows": moved, "dx": total}
        if s["residual"]:
            total += s["x"].double()
        return {"y": total, "dy": moved, "dw": dots} if s["grad"] else {"y": total}
    if op == "act_grad":
        return s["dy"].double() * _exact_act(s["z"].double(), s["act"], 1)
    if op == "linear":
        z = torch.mm(s["x"].double(), s["w"].double().t().contiguous())
        z += 0 if s["b"] is None else s["b"].double()
        y = _exact_act(z, s["act"], 0)
        y = y if s["r"] is None else y + s["r"].double()
        return {"y": y, "z": z} if s["keep"] else {"y": y}
    dz = s["dz"].double()
    dx = torch.mm(dz, s["w"].double()) * _exact_act(s["zx"].double(), s["act"], 1)
    dx = dx if s["add"] is None else dx + s["add"].double()
    return {"dx": dx, "dw": torch.mm(dz.t().contiguous(), s["x"].double()), "db": dz.sum(0)}
