"""The operators of the MXFP4 expert layer and of the router's training, as measured cases.

Each case is one pass through one operator; `op` names it:

* roundtrip  bf16 -> MXFP4 (32-element blocks, E8M0 scales, E2M1 codes) -> bf16
* gemm       the experts' product over MXFP4 activations and MXFP4 weights, rows grouped by expert
* dgrad      its input gradient through the dequantized weights, bf16 output gradients
* swiglu     SwiGLU forward that keeps its input in 8 bits, then its backward from those 8 bits
* router     balance loss, z-loss and per-expert counts, then the gradient of the logits

`own` selects the framework's kernels; otherwise `run` computes the plain form in elementary torch operations.
"""
import math

import torch

own = False

DEV = "cuda"
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one decoded token's hidden state, and a stack of expert matrices as a loader converts it
        {"name": "roundtrip one token", "op": "roundtrip", "mats": 1, "rows": 1, "cols": 6144},
        {"name": "roundtrip expert stack", "op": "roundtrip", "mats": 48, "rows": 4096, "cols": 6144},
        # gate/up product of one decoded token, top 8 of 256 experts
        {"name": "gemm decode one token", "op": "gemm", "E": 256, "k": 8, "T": 1, "N": 4096, "K": 6144, "gather": True, "zipf": False},
        # a small serving batch on the down projection of a narrow expert, with popular and empty experts
        {"name": "gemm serving batch", "op": "gemm", "E": 128, "k": 8, "T": 37, "N": 2048, "K": 768, "gather": False, "zipf": True},
        # a short prefill with ragged experts and sizes that are no multiple of a tile
        {"name": "gemm ragged prefill", "op": "gemm", "E": 60, "k": 4, "T": 1111, "N": 2848, "K": 2080, "gather": True, "zipf": True},
        # gate/up product of a training batch over one device's share of the experts
        {"name": "gemm training batch", "op": "gemm", "E": 64, "k": 8, "T": 8192, "N": 4096, "K": 6144, "gather": True, "zipf": False},
        # fine-tuning on a few short sequences, and the gate/up gradient of a training batch
        {"name": "dgrad short batch", "op": "dgrad", "E": 128, "k": 8, "T": 203, "N": 2048, "K": 768, "gather": True, "zipf": True},
        {"name": "dgrad training batch", "op": "dgrad", "E": 64, "k": 8, "T": 8192, "N": 4096, "K": 6144, "gather": False, "zipf": False},
        # the activation between the two products: a few short sequences, and a training batch
        {"name": "swiglu short batch", "op": "swiglu", "T": 101, "k": 8, "I": 768},
        {"name": "swiglu training batch", "op": "swiglu", "T": 16384, "k": 8, "I": 2048},
        # router of a small layer on a padded batch; router of a large one over many sequences with masked experts
        {"name": "router padded batch", "op": "router", "T": 515, "E": 60, "k": 4, "renorm": True, "padded": True, "masked": 0},
        {"name": "router training batch", "op": "router", "T": 131072, "E": 256, "k": 8, "renorm": False, "padded": False, "masked": 16},
    ]


def _between(rng, lo, hi, step=1):
    """A multiple of step in [lo, hi], spread evenly over the logarithm."""
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi)))) // step * step))


def draw(rng):
    op = rng.choice(("roundtrip", "gemm", "gemm", "dgrad", "swiglu", "router"))
    if op == "roundtrip":
        return {"op": op, "mats": _between(rng, 1, 16), "rows": _between(rng, 1, 4096), "cols": _between(rng, 32, 8192, 32)}
    if op in ("gemm", "dgrad"):
        E = rng.choice((8, 16, 60, 64, 128))
        k = min(E, rng.choice((1, 2, 4, 6, 8)))
        T = _between(rng, 1 if op == "gemm" else 16, 4096)
        most = 1 << 42  # T k N K of a drawn case stays under the largest listed one's
        N, K = _between(rng, 128, 6144, 32), _between(rng, 128, 6144, 32)
        while T * k * N * K * 2 > most or E * N * K > 1 << 30:
            N, K = max(128, N // 64 * 32), max(128, K // 64 * 32)
        return {"op": op, "E": E, "k": k, "T": T, "N": N, "K": K, "gather": rng.random() < 0.5, "zipf": rng.random() < 0.5}
    if op == "swiglu":
        return {"op": op, "T": _between(rng, 1, 8192), "k": rng.choice((1, 2, 4, 8)), "I": _between(rng, 32, 4096, 32)}
    E = rng.choice((8, 16, 37, 60, 64, 128, 160, 256, 384, 512, 1000))
    return {"op": op, "T": _between(rng, 1, 32768), "E": E, "k": min(E, _between(rng, 1, 16)), "renorm": rng.random() < 0.5,
            "padded": rng.random() < 0.5, "masked": rng.choice((0, 0, E // 16))}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed) * 1_000_003 + 17)


def _normal(g, shape, std):
    return torch.randn(shape, generator=g, device=DEV).mul_(std).to(torch.bfloat16)


def _outliers(g, x):
    """Values as weights and activations have them: one in a thousand twenty times as large."""
    return torch.where(torch.rand(x.shape, generator=g, device=DEV) < 0.001, x * 20, x)


def _codes(x):
    """MXFP4 codes (two per byte, even element low) and scales of bf16 rows, as a model file holds them."""
    b = x.float().unflatten(-1, (-1, 32))
    amax = b.abs().amax(-1, keepdim=True)
    s = torch.where(amax > 0, torch.frexp(amax).exponent - 3, -127).clamp(-127, 125)
    mag = torch.bucketize((b * torch.exp2(-s.float())).abs(), torch.tensor((0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0), device=DEV)).to(torch.uint8)
    c = (mag | (torch.signbit(b).to(torch.uint8) << 3)).flatten(-2)
    return c[..., 0::2] | (c[..., 1::2] << 4), (s.squeeze(-1) + 127).to(torch.uint8)


def _stack(g, E, N, K):
    codes = torch.empty((E, N, K // 2), dtype=torch.uint8, device=DEV)
    scales = torch.empty((E, N, K // 32), dtype=torch.uint8, device=DEV)
    step = max(1, (1 << 27) // (N * K))
    for e in range(0, E, step):
        n = min(step, E - e)
        codes[e:e + n], scales[e:e + n] = _codes(_outliers(g, _normal(g, (n, N, K), 0.02)))
    return codes, scales


def _routing(g, T, E, k, zipf):
    """k experts for each token, and the routed pairs in order of their expert, as the framework's permutation gives them."""
    score = -torch.log(-torch.log(torch.rand((T, E), generator=g, device=DEV).clamp(1e-7, 1 - 1e-7)))
    if zipf:  # popular and unpopular experts; one in sixteen gets no token
        rank = torch.randperm(E, generator=g, device=DEV)
        score = score - 1.1 * torch.log(rank + 1.0)
        score[:, rank > max(k, E - E // 16) - 1] = float("-inf")
    idx = score.topk(k, dim=1).indices
    flat = idx.flatten()
    perm = torch.argsort(flat, stable=True)
    counts = torch.zeros(E, dtype=torch.int64, device=DEV).scatter_add_(0, flat, torch.ones_like(flat))
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    return {"perm": perm.int(), "offsets": offsets.int(), "counts": counts, "expert": flat[perm]}


def prepare(case, seed):
    c, g = dict(case), _gen(seed)
    op = c["op"]
    if op == "roundtrip":
        x = torch.empty((c["mats"], c["rows"], c["cols"]), dtype=torch.bfloat16, device=DEV)
        for m in range(c["mats"]):
            x[m] = _outliers(g, _normal(g, x.shape[1:], 0.02))
        return {**c, "x": x, "y": torch.empty_like(x), "codes": torch.empty((*x.shape[:2], c["cols"] // 2), dtype=torch.uint8, device=DEV),
                "scales": torch.empty((*x.shape[:2], c["cols"] // 32), dtype=torch.uint8, device=DEV)}
    if op in ("gemm", "dgrad"):
        T, E, k, N, K = c["T"], c["E"], c["k"], c["N"], c["K"]
        R = T * k
        s = {**c, **_routing(g, T, E, k, c["zipf"]), "R": R}
        s["w_codes"], s["w_scales"] = _stack(g, E, N, K)
        rows = T if c["gather"] else R
        # the plan of the plain form: the experts that have rows, padded to the most rows one has
        s["hit"] = torch.nonzero(s["counts"]).flatten()
        s["cap"] = int(s["counts"].max())
        place = torch.zeros(E, dtype=torch.int64, device=DEV)
        place[s["hit"]] = torch.arange(s["hit"].numel(), device=DEV)
        s["dest"] = place[s["expert"]] * s["cap"] + torch.arange(R, device=DEV) - s["offsets"].long()[s["expert"]]
        s["src"] = s["perm"].long() // k if c["gather"] else torch.arange(R, device=DEV)
        if op == "gemm":
            x = _outliers(g, _normal(g, (1, rows, K), 1.0))
            s["x_codes"], s["x_scales"] = _codes(x)
            s["y"] = torch.empty((R, N), dtype=torch.bfloat16, device=DEV)
        else:
            s["dy"] = _normal(g, (rows, N), 1.0)
            s["dx"] = torch.empty((R, K), dtype=torch.bfloat16, device=DEV)
        return s
    if op == "swiglu":
        R, I = c["T"] * c["k"], c["I"]
        s = {**c, "R": R, "h": _outliers(g, _normal(g, (R, 2 * I), 1.0)), "da": _normal(g, (R, I), 1.0),
             "perm": torch.randperm(R, generator=g, device=DEV).int(), "w": torch.rand((c["T"], c["k"]), generator=g, device=DEV)}
        s["h8"] = torch.empty((R, 2 * I), dtype=torch.uint8, device=DEV)
        s["h8_scales"] = torch.empty((R, 2 * I // 32), dtype=torch.uint8, device=DEV)
        s["a"] = torch.empty((R, I), dtype=torch.bfloat16, device=DEV)
        s["dh"] = torch.empty((R, 2 * I), dtype=torch.bfloat16, device=DEV)
        s["dw"] = torch.empty((c["T"], c["k"]), device=DEV)
        return s
    T, E, k = c["T"], c["E"], c["k"]
    logits = torch.randn((T, E), generator=g, device=DEV) + torch.randn(E, generator=g, device=DEV)
    if c["masked"]:  # experts that are switched off
        off = torch.randperm(E, generator=g, device=DEV)[: min(c["masked"], E - k)]
        logits[:, off] = float("-inf")
    s = {**c, "idx": logits.topk(k, dim=1).indices.int(), "dw": torch.randn((T, k), generator=g, device=DEV) / T,
         "dloss": torch.tensor((0.01, 0.001), device=DEV)}
    valid = torch.ones(T, dtype=torch.uint8, device=DEV)
    if c["padded"] and T > 1:  # padding holds whatever its rows came out as
        pad = torch.rand(T, generator=g, device=DEV) < 0.2
        pad[0] = False
        valid[pad] = 0
        logits[pad] = float("nan")
        s["dw"][pad] = float("nan")
    s["valid"] = valid if c["padded"] else None
    s["logits"] = logits
    s["counts"] = torch.empty(E + 1, dtype=torch.int32, device=DEV)
    s["loss"] = torch.empty(2, device=DEV)
    s["dlogits"] = torch.empty((T, E), device=DEV)
    s["ws"] = torch.empty(1 << 22, dtype=torch.uint8, device=DEV)
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _two_to(e):
    return torch.ldexp(torch.ones_like(e, dtype=torch.float32), e)


def _plain_roundtrip(x):
    b = x.float().unflatten(-1, (-1, 32))
    amax = b.abs().amax(-1, keepdim=True)
    s = torch.where(amax > 0, torch.frexp(amax).exponent - 3, -127).clamp(-127, 125)
    v = b * _two_to(-s)
    m = v.abs()
    q = torch.where(m < 2, torch.round(2 * m) / 2, torch.where(m < 4, torch.round(m), 2 * torch.round(m / 2))).clamp(max=6)
    return (torch.copysign(q, v) * _two_to(s)).flatten(-2).to(x.dtype)


def _values(codes, scales):
    """The float32 values of MXFP4 rows."""
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
    both = torch.arange(256, device=codes.device)
    pairs = torch.stack([table[both & 15], table[both >> 4]], -1)
    v = pairs.index_select(0, codes.flatten().int()).view(*scales.shape, 32)
    return (v * _two_to(scales.int().unsqueeze(-1) - 127)).flatten(-2)


def _plain_gemm(s):
    w = _values(s["w_codes"][s["hit"]], s["w_scales"][s["hit"]])
    x = _values(s["x_codes"][0], s["x_scales"][0])
    xp = x.new_zeros((s["hit"].numel() * s["cap"], s["K"]))
    xp[s["dest"]] = x[s["src"]]
    y = torch.bmm(xp.view(-1, s["cap"], s["K"]), w.transpose(1, 2))
    return y.view(-1, s["N"])[s["dest"]].to(torch.bfloat16)


def _plain_dgrad(s):
    w = _values(s["w_codes"][s["hit"]], s["w_scales"][s["hit"]])
    dp = w.new_zeros((s["hit"].numel() * s["cap"], s["N"]))
    dp[s["dest"]] = s["dy"].float()[s["src"]]
    dx = torch.bmm(dp.view(-1, s["cap"], s["N"]), w)
    return dx.view(-1, s["K"])[s["dest"]].to(torch.bfloat16)


def _plain_eight_bits(h):
    """Values of the 8-bit copy: E4M3 in 32-element blocks, the smallest power of two that keeps a block within 448."""
    b = h.unflatten(-1, (-1, 32))
    m, e = torch.frexp(b.abs().amax(-1, keepdim=True))
    s = torch.where(m == 0, -127, torch.where(m <= 0.875, e - 9, e - 8)).clamp(-127, 127)
    v = b * _two_to(-s)
    step = _two_to(torch.frexp(v).exponent.clamp(min=-5) - 4)
    return (torch.round(v / step) * step * _two_to(s)).flatten(-2)


def _plain_swiglu(s):
    I = s["I"]
    h = s["h"].float()
    a = (h[:, :I] / (1 + torch.exp(-h[:, :I])) * h[:, I:]).to(torch.bfloat16)
    h = _plain_eight_bits(h)
    gate, up = h[:, :I], h[:, I:]
    da = s["da"].float()
    sig = 1 / (1 + torch.exp(-gate))
    perm = s["perm"].long()
    dw = torch.empty_like(s["w"]).flatten()
    dw[perm] = (da * gate * sig * up).sum(-1)
    da = da * s["w"].flatten()[perm].unsqueeze(-1)
    dh = torch.cat([da * up * sig * (1 + gate * (1 - sig)), da * gate * sig], -1)
    return {"a": a, "dh": dh.to(torch.bfloat16), "dw": dw.view_as(s["w"])}


def _plain_router(s):
    E, k = s["E"], s["k"]
    valid = torch.ones_like(s["logits"][:, 0], dtype=torch.bool) if s["valid"] is None else s["valid"] != 0
    l = torch.where(valid.unsqueeze(-1), s["logits"], 0.0)
    n = valid.sum()
    m = l.amax(-1, keepdim=True)
    ex = torch.exp(l - m)
    total = ex.sum(-1, keepdim=True)
    p, lse = ex / total, (m + torch.log(total)).squeeze(-1)
    idx = s["idx"].long()
    counts = torch.zeros(E, dtype=torch.int64, device=l.device).scatter_add_(0, idx.flatten(), valid.long().unsqueeze(-1).expand_as(idx).flatten())
    f = counts.double() / (n * k)
    mean = torch.where(valid.unsqueeze(-1), p, 0.0).sum(0, dtype=torch.float64) / n
    loss = torch.stack([E * (f * mean).sum(), torch.where(valid, lse, 0.0).double().square().sum() / n])
    # gradients
    g = s["dloss"]
    f = f.float()
    d = g[0] * E / n * (f - (p * f).sum(-1, keepdim=True)) * p + 2 * g[1] / n * lse.unsqueeze(-1) * p
    pw = p.gather(1, idx)
    dw = torch.where(valid.unsqueeze(-1), s["dw"], 0.0)
    if s["renorm"]:
        w = pw / pw.sum(-1, keepdim=True)
        d = d.scatter_add(1, idx, w * (dw - (w * dw).sum(-1, keepdim=True)))
    else:
        d = (d - (pw * dw).sum(-1, keepdim=True) * p).scatter_add(1, idx, pw * dw)
    d = torch.where(valid.unsqueeze(-1), d, 0.0)
    return {"counts": torch.cat([counts, n.unsqueeze(0)]).int(), "loss": loss.float(), "dlogits": d}


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def _own(s):
    import bit_quantized_moe_amd as bqm
    op = s["op"]
    if op == "roundtrip":
        q = bqm.QTensor(bqm.FMT_MXFP4, 0, s["mats"], s["rows"], s["cols"], s["codes"], s["scales"])
        bqm.bqm_quantize_mxfp4(s["x"], q)
        return bqm.bqm_dequantize(q, s["y"])
    if op in ("gemm", "dgrad"):
        w = bqm.QTensor(bqm.FMT_MXFP4, 0, s["E"], s["N"], s["K"], s["w_codes"], s["w_scales"])
        perm = s["perm"] if s["gather"] else None
        if op == "gemm":
            x = bqm.QTensor(bqm.FMT_MXFP4, 0, 1, s["x_codes"].shape[1], s["K"], s["x_codes"], s["x_scales"])
            return bqm.bqm_mxfp4_gemm(x, w, s["offsets"], perm, s["k"], s["y"])
        return bqm.bqm_mxfp4_dgrad(w, s["dy"], s["offsets"], perm, s["k"], s["dx"])
    if op == "swiglu":
        bqm.bqm_swiglu_ckpt_fwd(s["h"], s["h8"], s["h8_scales"], a=s["a"])
        bqm.bqm_swiglu_ckpt_bwd(s["h8"], s["h8_scales"], s["da"], s["perm"], s["w"], s["dh"], s["dw"])
        return {"a": s["a"], "dh": s["dh"], "dw": s["dw"]}
    bqm.bqm_router_loss(s["logits"], s["idx"], s["valid"], s["counts"], s["loss"], s["ws"])
    bqm.bqm_router_grad(s["logits"], s["idx"], s["valid"], s["counts"], s["dw"], s["dloss"], s["renorm"], s["dlogits"])
    return {"counts": s["counts"], "loss": s["loss"], "dlogits": s["dlogits"]}


def run(state):
    if own:
        return _own(state)
    op = state["op"]
    if op == "roundtrip":
        return _plain_roundtrip(state["x"])
    return {"gemm": _plain_gemm, "dgrad": _plain_dgrad, "swiglu": _plain_swiglu, "router": _plain_router}[op](state)


def work(case):
    c = case
    op = c["op"]
    if op == "roundtrip":  # input, codes and scales written and read, output
        n = c["mats"] * c["rows"] * c["cols"]
        return {"bytes": n * (2 + 2 * 17 / 32 + 2), "flops": 0}
    if op in ("gemm", "dgrad"):  # the weights of the experts that have rows, once
        T, E, k, N, K = (c[n] for n in ("T", "E", "k", "N", "K"))
        R = T * k
        hit = E * (1 - (1 - k / E) ** T)
        rows = T if c["gather"] else R
        moved = rows * K * 17 / 32 + R * N * 2 if op == "gemm" else rows * N * 2 + R * K * 2
        return {"bytes": hit * N * K * 17 / 32 + moved + 4 * (R * c["gather"] + E + 1), "flops": 2 * R * N * K}
    if op == "swiglu":  # h, a, the 8-bit copy written and read, da, dh
        n = c["T"] * c["k"] * c["I"]
        return {"bytes": n * (4 + 2 + 2 * 2 * 33 / 32 + 2 + 4) + 12 * c["T"] * c["k"], "flops": 30 * n}
    n = c["T"] * c["E"]  # the logits once for each direction, their gradient
    return {"bytes": 12 * n + 12 * c["T"] * c["k"] + c["T"] * (2 if c["padded"] else 0), "flops": 24 * n}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _nearest(v, grid):
    """The nearest value of an ascending grid of non-negative values, ties to the even place, for v >= 0."""
    mid = (grid[1:] + grid[:-1]) / 2
    lo, hi = torch.bucketize(v, mid), torch.bucketize(v, mid, right=True)
    at = torch.where(lo == hi, lo, torch.where(lo % 2 == 0, lo, hi))
    return grid[at]


def _exact_blocks(x, grid, exponent):
    b = x.double().unflatten(-1, (-1, 32))
    scale = exponent(b.abs().amax(-1, keepdim=True)).clamp(-127, 127).double().exp2()
    return (torch.sign(b) * _nearest((b / scale).abs(), grid) * scale).flatten(-2)


def _exact_weights(codes, scales):
    low, high = codes & 15, codes >> 4
    c = torch.stack([low, high], -1).flatten(-2).unflatten(-1, (-1, 32))
    mag = (c & 7).double()
    mag = torch.where(mag < 2, mag / 2, (1 + (mag % 2) / 2) * torch.floor(mag / 2 - 1).exp2())
    return ((1 - 2 * (c >> 3).double()) * mag * (scales.double().unsqueeze(-1) - 127).exp2()).flatten(-2)


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op == "roundtrip":
        grid = torch.tensor(E2M1, dtype=torch.float64, device=DEV)
        power = lambda a: torch.where(a > 0, torch.floor(torch.log2(a)) - 2, torch.full_like(a, -127.0))  # noqa: E731
        return torch.stack([_exact_blocks(x, grid, power) for x in s["x"]])
    if op in ("gemm", "dgrad"):
        out = torch.empty((s["R"], s["N"] if op == "gemm" else s["K"]), dtype=torch.float64, device=DEV)
        rows = _exact_weights(s["x_codes"][0], s["x_scales"][0]) if op == "gemm" else s["dy"].double()
        if s["gather"]:
            rows = rows[torch.div(s["perm"].long(), s["k"], rounding_mode="floor")]
        at = s["offsets"].tolist()
        for e in range(s["E"]):
            if at[e + 1] > at[e]:
                w = _exact_weights(s["w_codes"][e], s["w_scales"][e])
                out[at[e]:at[e + 1]] = rows[at[e]:at[e + 1]] @ (w.T.contiguous() if op == "gemm" else w)
        return out
    if op == "swiglu":
        I = s["I"]
        h = s["h"].double()
        a = h[:, :I] * torch.sigmoid(h[:, :I]) * h[:, I:]
        small = [m * 2.0 ** -9 for m in range(8)]
        grid = torch.tensor(small + [(8 + m) / 8 * 2.0 ** e for e in range(-6, 9) for m in range(8) if (e, m) != (8, 7)], dtype=torch.float64, device=DEV)
        least = lambda t: torch.where(t > 0, torch.ceil(torch.log2(t / 448)), torch.full_like(t, -127.0))  # noqa: E731
        h = _exact_blocks(s["h"], grid, least)
        gate, up, da = h[:, :I], h[:, I:], s["da"].double()
        sig = torch.sigmoid(gate)
        flat = s["perm"].long()
        dw = torch.zeros(s["R"], dtype=torch.float64, device=DEV).index_copy(0, flat, torch.linalg.vecdot(da, gate * sig * up))
        w = s["w"].double().flatten()[flat].unsqueeze(-1)
        dh = torch.cat([w * da * up * (sig + gate * sig * (1 - sig)), w * da * gate * sig], -1)
        return {"a": a, "dh": dh, "dw": dw.view_as(s["w"])}
    E, k, g = s["E"], s["k"], s["dloss"].double()
    keep = torch.arange(s["T"], device=DEV) if s["valid"] is None else torch.nonzero(s["valid"]).flatten()
    l, idx, dw = s["logits"][keep].double(), s["idx"][keep].long(), s["dw"][keep].double()
    n = keep.numel()
    p, lse = torch.softmax(l, -1), torch.logsumexp(l, -1)
    counts = torch.stack([(idx == e).sum() for e in range(E)])
    f, mean = counts.double() / (n * k), p.mean(0)
    loss = torch.stack([E * (f @ mean), lse.square().mean()])
    up = (g[0] * E / n) * f.expand(n, E)  # the gradient of the probabilities
    pw = p.gather(1, idx)
    total = pw.sum(1, keepdim=True) if s["renorm"] else torch.ones_like(pw[:, :1])
    dpw = (dw - ((pw * dw).sum(1, keepdim=True) / total if s["renorm"] else 0)) / total
    up = up.scatter_add(1, idx, dpw)
    d = p * (up - (p * up).sum(1, keepdim=True)) + (2 * g[1] / n) * lse.unsqueeze(1) * p
    out = torch.zeros_like(s["logits"], dtype=torch.float64)
    out[keep] = d
    return {"counts": torch.cat([counts, counts.new_tensor([n])]).int(), "loss": loss, "dlogits": out}
