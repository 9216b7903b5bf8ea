"""Cases of the operators around the layer in a language-model training step: routing by scores, layer norm,
token embedding and distillation from a teacher's top logits.  `run` computes a case in plain torch operations,
or, where `own` is true, with the library's kernels."""

import math

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
MASKED, LEFT_OUT = -1e300, -math.inf  # ranks of a masked expert, and of one outside the kept groups


# ---- cases


def _route(name, N, E, k, score, bias, groups, kept, renorm, scale, masked, back):
    return {"name": name, "op": "route", "N": N, "E": E, "k": k, "score": score, "bias": bias, "groups": groups, "kept": kept, "group_top": 2,
            "renorm": renorm, "scale": scale, "masked": masked, "back": back}


def _lnorm(name, N, H, dtype, way):
    return {"name": name, "op": "lnorm", "N": N, "H": H, "dtype": dtype, "way": way}


def _embed(name, N, V, H, dtype, way):
    return {"name": name, "op": "embed", "N": N, "V": V, "H": H, "dtype": dtype, "way": way}


def _distill(name, N, H, V, v_chunk, K, T):
    return {"name": name, "op": "distill", "N": N, "H": H, "V": V, "v_chunk": v_chunk, "K": K, "T": T}


def listed():
    return [
        # one token of a served model: sigmoid scores, a balance bias, 4 of 8 groups kept; latency is all there is
        _route("route_one_token", 1, 256, 8, "sigmoid", True, 8, 4, True, 2.5, False, False),
        # a training batch of the layer's 64-expert configuration, softmax gates renormalised, with the gradient
        _route("route_64_experts", 65536, 64, 8, "softmax", False, 1, 1, True, 1.0, False, True),
        # a training batch over 256 experts in groups with a balance bias, with the gradient
        _route("route_grouped", 16384, 256, 8, "sigmoid", True, 8, 4, True, 2.5, False, True),
        # the layer's 896-expert configuration, softmax scores as they are: the gradient reaches every expert
        _route("route_896_experts", 8192, 896, 16, "softmax", False, 1, 1, False, 1.0, True, True),
        # one token's hidden row
        _lnorm("lnorm_one_token", 1, 2048, "bf16", "fwd"),
        # the 65,536-token training batch, forward and backward
        _lnorm("lnorm_train", 65536, 2048, "bf16", "both"),
        # wide rows of the vocabulary workload
        _lnorm("lnorm_wide_back", 8192, 7168, "bf16", "bwd"),
        # a ragged batch of rows that no vector width divides, in 32 bits
        _lnorm("lnorm_odd_f32", 777, 1111, "f32", "both"),
        # the lookup in front of a training step, over the 200,000-entry vocabulary
        _embed("embed_lookup", 8192, 200_000, 7168, "bf16", "fwd"),
        # its gradient for the 65,536-token batch: text's skew, one token in 18 being the commonest
        _embed("embed_train_back", 65536, 200_000, 2048, "bf16", "bwd"),
        # a small ragged distillation batch: short last strip, short last tiles
        _distill("distill_small", 777, 512, 20_000, 4096, 16, 2.0),
        # the vocabulary workload's projection under a teacher's 32 best logits
        _distill("distill_vocab", 8192, 7168, 200_000, 8192, 32, 1.0),
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["route", "lnorm", "embed", "distill"])
    if op == "route":
        N, E = _spread(rng, 1, 65536), rng.choice([8, 60, 64, 72, 128, 160, 256, 384, 512, 896, 1000, 1024])
        N = max(1, min(N, 16_777_216 // E))
        g = rng.choice([n for n in (1, 1, 2, 4, 8) if E % n == 0 and E // n >= 4])
        kept = rng.randint(1, g)
        k = _spread(rng, 1, min(32, kept * (E // g)))
        score = rng.choice(["softmax", "sigmoid"])
        c = _route("", N, E, k, score, rng.random() < 0.5, g, kept, rng.random() < 0.6, rng.choice([1.0, 2.5]), rng.random() < 0.3, rng.random() < 0.7)
        c["group_top"] = rng.choice([1, 2])
    elif op == "lnorm":
        N, H = _spread(rng, 1, 65536), _spread(rng, 64, 12000)
        if rng.random() < 0.7:
            H = -(-H // 64) * 64
        c = _lnorm("", max(1, min(N, 134_217_728 // H)), H, rng.choice(["bf16", "bf16", "f32"]), rng.choice(["fwd", "bwd", "both"]))
    elif op == "embed":
        H, V = _spread(rng, 64, 7168), _spread(rng, 100, 200_000)
        if rng.random() < 0.8:
            H = -(-H // 64) * 64
        V = min(V, 409_600_000 // H)
        N = min(_spread(rng, 1, 65536), 134_217_728 // H)
        c = _embed("", N, V, H, rng.choice(["bf16", "bf16", "f32"]), rng.choice(["fwd", "bwd"]))
    else:
        N, H, V = _spread(rng, 16, 8192), 128 * _spread(rng, 1, 56), _spread(rng, 300, 200_000)
        V = max(300, min(V, 1_500_000_000_000 // (N * H)))
        c = _distill("", N, H, V, 256 * _spread(rng, 4, 64), _spread(rng, 1, 64), rng.choice([1.0, 2.0, 4.0]))
    del c["name"]
    return c


# ---- inputs


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    s = {"case": c}

    def normal(*shape, std=1.0, dtype=torch.float32):
        # in slabs, so that a large matrix needs no 32-bit copy of itself
        out = torch.empty(shape, dtype=dtype, device=DEV)
        rows = max(1, (1 << 26) // max(1, math.prod(shape[1:])))
        for r in range(0, shape[0], rows):
            part = out[r:r + rows]
            part.copy_(torch.randn(part.shape, generator=g, device=DEV).mul_(std))
        return out

    if c["op"] == "route":
        N, E, k = c["N"], c["E"], c["k"]
        s["logits"] = normal(N, E, std=1.2)
        if c["masked"]:  # a twentieth of the experts is away for each token
            s["logits"][torch.rand((N, E), generator=g, device=DEV) < 0.05] = -math.inf
        s["bias"] = normal(E, std=0.1) if c["bias"] else None
        s["dgates"] = normal(N, k) if c["back"] else None
        if own:
            from memory_bounded_expert_amd import binding as B
            s["plan"] = B.route_plan(N, E, k, score=c["score"], n_group=c["groups"], topk_group=c["kept"], group_top=c["group_top"],
                                     renorm=c["renorm"], scale=c["scale"])
    elif c["op"] == "lnorm":
        N, H, dt = c["N"], c["H"], DTYPES[c["dtype"]]
        # hidden rows: channels with means and widths of their own
        x = normal(N, H) * (0.5 + torch.rand(H, generator=g, device=DEV)) + normal(H, std=0.3)
        s["X"] = x.to(dt)
        s["gamma"], s["beta"], s["eps"] = 1 + normal(H, std=0.1), normal(H, std=0.1), 1e-5
        if c["way"] != "fwd":
            s["dY"] = normal(N, H, dtype=dt)
        if c["way"] == "bwd":  # what the forward pass has kept
            x = s["X"].double()
            m = x.mean(1)
            s["mean"], s["rstd"] = m.float(), ((x - m[:, None]).square().mean(1) + s["eps"]).rsqrt().float()
        if own:
            from memory_bounded_expert_amd import binding as B
            s["plan"] = B.lnorm_plan(N, H, B.moe_dtype(dt), s["eps"])
            s["ws"] = B.workspace(s["plan"], "bwd", torch.device("cuda:0")) if c["way"] != "fwd" else None
    elif c["op"] == "embed":
        N, V, H, dt = c["N"], c["V"], c["H"], DTYPES[c["dtype"]]
        # ranks follow 1/r as words do, scattered over the table; one position in 50 is padding
        r = torch.rand(N, generator=g, device=DEV, dtype=torch.float64).mul_(math.log(V)).exp_().long().sub_(1).clamp_(0, V - 1)
        ids = (r * 7919 + 13) % V
        ids[torch.rand(N, generator=g, device=DEV) < 0.02] = -1
        s["ids"], s["scale"] = ids.int(), math.sqrt(H)
        if c["way"] == "fwd":
            s["W"] = normal(V, H, std=0.02, dtype=dt)
        else:
            s["dY"] = normal(N, H, dtype=dt)
        if own:
            from memory_bounded_expert_amd import binding as B
            s["plan"] = B.embed_plan(N, V, H, B.moe_dtype(dt), s["scale"])
            s["ws"] = B.workspace(s["plan"], "bwd", torch.device("cuda:0")) if c["way"] != "fwd" else None
    else:
        N, H, V, K = c["N"], c["H"], c["V"], c["K"]
        s["X"], s["W"] = normal(N, H, dtype=torch.bfloat16), normal(V, H, std=0.02, dtype=torch.bfloat16)
        # the teacher's best entries, all different; some lists are shorter, some positions are padding
        step = V // K
        at = torch.randint(0, V, (N, 1), generator=g, device=DEV) + torch.arange(K, device=DEV) * step
        at = (at + torch.randint(0, step, (N, K), generator=g, device=DEV)) % V
        best = (8 + 2 * normal(N, K)).sort(1, descending=True).values
        size = torch.where(torch.rand(N, generator=g, device=DEV) < 0.1, torch.randint(0, K + 1, (N,), generator=g, device=DEV), K)
        at[torch.arange(K, device=DEV) >= size[:, None]] = -1
        s["t_idx"], s["t_logit"] = at.int(), best
        s["dloss"] = (0.5 + torch.rand(N, generator=g, device=DEV)) / N
        if own:
            from memory_bounded_expert_amd import binding as B
            s["plan"] = B.kd_plan(N, H, V, c["v_chunk"], K, c["T"], dw_dtype=B.MOE_BF16)
            s["ws"] = B.workspace(s["plan"], "both", torch.device("cuda:0"))
    return s


# ---- one pass


def run(s):
    return {"route": _run_route, "lnorm": _run_lnorm, "embed": _run_embed, "distill": _run_distill}[s["case"]["op"]](s)


def _run_route(s):
    c, lg = s["case"], s["logits"]
    if own:
        from memory_bounded_expert_amd import binding as B
        idx, gates = B.route_forward(s["plan"], lg, s["bias"])
        if not c["back"]:
            return {"idx": idx, "gates": gates}
        return {"idx": idx, "gates": gates, "dlogits": B.route_backward(s["plan"], lg, idx, s["dgates"])}
    N, E = lg.shape
    k, g = c["k"], c["groups"]
    l = lg.double()  # which of two near scores is larger shows in 64 bits
    if c["score"] == "sigmoid":
        score = 1 / (1 + torch.exp(-l))
    else:
        score = torch.exp(l - l.amax(1, keepdim=True))
        score = score / score.sum(1, keepdim=True)
    gone = l == -math.inf
    key = score + s["bias"].double() if c["bias"] else score
    rank = (key if c["bias"] else l).masked_fill(gone, MASKED)  # without a bias the logits' order is the scores'
    if g > 1:
        best = key.masked_fill(gone, -math.inf).view(N, g, E // g).sort(2, descending=True).values[:, :, :c["group_top"]]
        total = torch.where(best == -math.inf, 0.0, best).sum(2).masked_fill(best[:, :, 0] == -math.inf, -math.inf)
        keep = total.sort(dim=1, descending=True, stable=True).indices[:, :c["kept"]]
        kept = torch.zeros((N, g), dtype=torch.bool, device=lg.device).scatter_(1, keep, True)
        rank = rank.view(N, g, E // g).masked_fill(~kept[:, :, None], LEFT_OUT).view(N, E)
    idx = rank.sort(dim=1, descending=True, stable=True).indices[:, :k]
    sel = score.gather(1, idx)
    total = sel.sum(1, keepdim=True) if c["renorm"] else 1.0
    part = torch.where(sel > 0, sel / total, 0.0)
    gates = c["scale"] * part
    out = {"idx": idx.int(), "gates": gates.float()}
    if c["back"]:
        dg = s["dgates"].double()
        dot = (gates * dg).sum(1, keepdim=True)
        if c["score"] == "sigmoid":
            d = part * (1 - sel) * ((c["scale"] * dg - dot) if c["renorm"] else c["scale"] * dg)
            dl = torch.zeros_like(l).scatter_(1, idx, d)
        elif c["renorm"]:
            dl = torch.zeros_like(l).scatter_(1, idx, part * (c["scale"] * dg - dot))
        else:
            dl = (-score * dot).scatter_add_(1, idx, gates * dg)
        out["dlogits"] = dl.float()
    return out


def _run_lnorm(s):
    way, out = s["case"]["way"], {}
    if own:
        from memory_bounded_expert_amd import binding as B
        mean, rstd = s.get("mean"), s.get("rstd")
        if way != "bwd":
            out["Y"], mean, rstd = B.lnorm_forward(s["plan"], s["X"], s["gamma"], s["beta"])
            out["mean"], out["rstd"] = mean, rstd
        if way != "fwd":
            out["dX"], out["dgamma"], out["dbeta"] = B.lnorm_backward(s["plan"], s["X"], s["gamma"], s["dY"], mean, rstd, ws=s["ws"])
        return out
    x = s["X"].float()
    if way == "bwd":
        mean, rstd = s["mean"], s["rstd"]
    else:
        mean = x.mean(1)
        rstd = ((x - mean[:, None]).square().mean(1) + s["eps"]).rsqrt()
        out["mean"], out["rstd"] = mean, rstd
    xhat = (x - mean[:, None]) * rstd[:, None]
    if way != "bwd":
        out["Y"] = (xhat * s["gamma"] + s["beta"]).to(s["X"].dtype)
    if way != "fwd":
        dy = s["dY"].float()
        d = dy * s["gamma"]
        dx = rstd[:, None] * (d - d.mean(1, keepdim=True) - xhat * (d * xhat).mean(1, keepdim=True))
        out["dX"], out["dgamma"], out["dbeta"] = dx.to(s["X"].dtype), (dy * xhat).sum(0), dy.sum(0)
    return out


def _run_embed(s):
    c, ids = s["case"], s["ids"]
    if own:
        from memory_bounded_expert_amd import binding as B
        if c["way"] == "fwd":
            return {"Y": B.embed_forward(s["plan"], s["W"], ids)}
        return {"dW": B.embed_backward(s["plan"], ids, s["dY"], ws=s["ws"])}
    real = (ids >= 0) & (ids < c["V"])
    at = torch.where(real, ids, 0).long()
    if c["way"] == "fwd":
        y = s["W"][at].float() * s["scale"]
        return {"Y": torch.where(real[:, None], y, 0.0).to(s["W"].dtype)}
    d = torch.where(real[:, None], s["dY"].float(), 0.0)
    dW = torch.zeros((c["V"], c["H"]), dtype=torch.float32, device=ids.device).index_add_(0, at, d)
    return {"dW": dW.mul_(s["scale"])}


def _run_distill(s):
    c, X, W = s["case"], s["X"], s["W"]
    if own:
        from memory_bounded_expert_amd import binding as B
        loss, lse, y_top = B.kd_forward(s["plan"], X, W, s["t_idx"], s["t_logit"], ws=s["ws"])
        dX, dW = B.kd_backward(s["plan"], X, W, s["t_idx"], s["t_logit"], lse, y_top, s["dloss"], ws=s["ws"])
        return {"loss": loss, "lse": lse, "y_top": y_top, "dX": dX, "dW": dW}
    T, V = c["T"], c["V"]
    x, w = X.float(), W.float()
    y = x @ w.T
    real = (s["t_idx"] >= 0) & (s["t_idx"] < V)
    at = torch.where(real, s["t_idx"], 0).long()
    y_top = torch.where(real, y.gather(1, at), 0.0)
    t = (s["t_logit"] / T).masked_fill(~real, -math.inf)
    some = real.any(1, keepdim=True)
    top = torch.where(some, t.amax(1, keepdim=True), 0.0)
    p = torch.exp(t - top)
    z = torch.where(some, p.sum(1, keepdim=True), 1.0)
    p, logp = p / z, torch.where(real, t - top - z.log(), 0.0)
    y.mul_(1 / T)
    m = y.amax(1, keepdim=True)
    y.sub_(m).exp_()
    z = y.sum(1, keepdim=True)
    lse = (m + z.log())[:, 0]
    loss = T * T * (p * (logp - y_top / T + lse[:, None])).sum(1)
    y.div_(z).scatter_add_(1, at, -p)
    y.mul_(torch.where(some, s["dloss"][:, None] * T, 0.0))
    return {"loss": loss, "lse": lse, "y_top": y_top, "dX": (y @ w).to(X.dtype), "dW": (y.T @ x).to(W.dtype)}


# ---- what a pass cannot do without


def work(case):
    c, N = case, case["N"]
    if c["op"] == "route":
        E, k = c["E"], c["k"]
        moved = N * E * 4 + N * k * 8 + (E * 4 if c["bias"] else 0)
        if c["back"]:
            moved += N * E * 4 + N * k * 4  # dlogits written, dgates read; the logits are there already
        return {"bytes": moved, "flops": N * E * (8 if c["back"] else 4)}
    if c["op"] == "lnorm":
        H, b = c["H"], 2 if c["dtype"] == "bf16" else 4
        rows = {"fwd": 2, "bwd": 3, "both": 4}[c["way"]]
        return {"bytes": rows * N * H * b + 8 * N + 16 * H, "flops": N * H * {"fwd": 8, "bwd": 14, "both": 22}[c["way"]]}
    if c["op"] == "embed":
        H, V, b = c["H"], c["V"], 2 if c["dtype"] == "bf16" else 4
        if c["way"] == "fwd":
            seen = V * (1 - math.exp(-N / V)) if N < V else V  # at most these rows are read
            return {"bytes": N * 4 + N * H * b + int(seen) * H * b, "flops": N * H}
        return {"bytes": N * 4 + N * H * b + V * H * 4, "flops": N * H}
    H, V, K = c["H"], c["V"], c["K"]
    return {"bytes": 2 * N * H * 2 + 2 * V * H * 2 + N * K * 12 + N * 12, "flops": 6 * N * H * V}


# ---- the definitions in 64 bits


def exact(case, seed):
    c, s = dict(case), prepare(case, seed)
    return {"route": _exact_route, "lnorm": _exact_lnorm, "embed": _exact_embed, "distill": _exact_distill}[c["op"]](c, s)


def _exact_route(c, s):
    l = s["logits"].double()
    N, E = l.shape
    dev, g, per = l.device, c["groups"], E // c["groups"]
    logp = -torch.nn.functional.softplus(-l) if c["score"] == "sigmoid" else torch.log_softmax(l, 1)
    value = logp.exp()
    if c["bias"]:
        value = value + s["bias"].double()
    there = torch.isfinite(l)
    open_ = torch.ones((N, E), dtype=torch.bool, device=dev)
    if g > 1:
        strength = torch.full((N, g), -math.inf, dtype=torch.float64, device=dev)
        for j in range(g):
            v = torch.where(there, value, -math.inf)[:, j * per:(j + 1) * per].clone()
            total, any_ = torch.zeros(N, dtype=torch.float64, device=dev), torch.zeros(N, dtype=torch.bool, device=dev)
            for _ in range(c["group_top"]):
                best, where = v.max(1)
                has = best > -math.inf
                total, any_ = total + torch.where(has, best, 0.0), any_ | has
                v.scatter_(1, where[:, None], -math.inf)
            strength[:, j] = torch.where(any_, total, -math.inf)
        # a group is kept where fewer than `kept` groups come before it
        before = strength[:, None, :] > strength[:, :, None]
        same = (strength[:, None, :] == strength[:, :, None]) & (torch.arange(g, device=dev)[None, :] < torch.arange(g, device=dev)[:, None])
        open_ = ((before | same).sum(2) < c["kept"]).repeat_interleave(per, 1)
    left = torch.where(open_, torch.where(there, value if c["bias"] else l, -1e200), -math.inf)
    places = torch.arange(E, device=dev)
    idx = []
    for _ in range(c["k"]):
        at = torch.where(left == left.amax(1, keepdim=True), places, E).amin(1)
        idx.append(at)
        left.scatter_(1, at[:, None], -math.inf)
    idx = torch.stack(idx, 1)
    chosen = torch.zeros((N, E), dtype=torch.bool, device=dev).scatter_(1, idx, True)
    if c["renorm"]:
        z = torch.where(chosen, logp, -math.inf).logsumexp(1, keepdim=True)
        z = torch.where(torch.isfinite(z), z, 0.0)
        gate = torch.where(chosen, (logp - z).exp(), 0.0) * c["scale"]
    else:
        gate = torch.where(chosen, logp.exp(), 0.0) * c["scale"]
    out = {"idx": idx.int(), "gates": gate.gather(1, idx)}
    if c["back"]:
        up = torch.zeros((N, E), dtype=torch.float64, device=dev).scatter_(1, idx, s["dgates"].double())
        dlogp = gate * up  # through gate = scale exp(logp - z)
        if c["renorm"]:
            dlogp = dlogp - gate / c["scale"] * dlogp.sum(1, keepdim=True)
        if c["score"] == "sigmoid":
            out["dlogits"] = dlogp * torch.sigmoid(-l)
        else:
            out["dlogits"] = dlogp - logp.exp() * dlogp.sum(1, keepdim=True)
    return out


def _exact_lnorm(c, s):
    x, gamma, out = s["X"].double(), s["gamma"].double(), {}
    H = c["H"]
    if c["way"] == "bwd":
        mean, r = s["mean"].double()[:, None], s["rstd"].double()[:, None]
    else:
        mean = x.sum(1, keepdim=True) / H
        r = 1 / torch.sqrt((x * x).sum(1, keepdim=True) / H - mean * mean + s["eps"])
        out["mean"], out["rstd"] = mean[:, 0], r[:, 0]
        out["Y"] = torch.addcmul(s["beta"].double(), (x - mean) * r, gamma)
    if c["way"] != "fwd":
        dy = s["dY"].double()
        n = x.sub_(mean).mul_(r)
        a, b = dy @ gamma / H, ((dy * n) @ gamma) / H
        out["dgamma"], out["dbeta"] = torch.einsum("nh,nh->h", dy, n), torch.ones(1, len(dy), dtype=torch.float64, device=dy.device).matmul(dy)[0]
        out["dX"] = (dy * gamma - a[:, None] - n * b[:, None]) * r
    return out


def _exact_embed(c, s):
    ids = s["ids"].long()
    real = ((ids >= 0) & (ids < c["V"])).nonzero()[:, 0]
    if c["way"] == "fwd":
        y = torch.zeros((c["N"], c["H"]), dtype=torch.float64, device=ids.device)
        y[real] = s["W"].double().index_select(0, ids[real]) * s["scale"]
        return {"Y": y}
    dW = torch.zeros((c["V"], c["H"]), dtype=torch.float64, device=ids.device)
    dW.index_put_((ids[real],), s["dY"][real].double() * s["scale"], accumulate=True)
    return {"dW": dW}


def _exact_distill(c, s):
    N, H, V, T = c["N"], c["H"], c["V"], c["T"]
    x, dev = s["X"].double(), s["X"].device
    ok = (s["t_idx"] >= 0) & (s["t_idx"] < V)
    some = ok.any(1)
    t = torch.where(ok, s["t_logit"].double() / T, -math.inf)
    logp = torch.where(ok, torch.log_softmax(torch.where(some[:, None], t, 0.0), 1), -math.inf)
    p = logp.exp()
    at = torch.where(ok, s["t_idx"], 0).long()
    lse = torch.full((N,), -math.inf, dtype=torch.float64, device=dev)
    y_top = torch.zeros_like(p)
    blocks = [(v, min(V, v + 25_000)) for v in range(0, V, 25_000)]
    for v0, v1 in blocks:
        y = x @ s["W"][v0:v1].double().T
        lse = torch.logaddexp(lse, (y / T).logsumexp(1))
        here = ok & (at >= v0) & (at < v1)
        y_top = torch.where(here, y.gather(1, (at - v0).clamp(0, v1 - v0 - 1)), y_top)
    loss = T * T * torch.where(ok, p * (logp - (y_top / T - lse[:, None])), 0.0).sum(1)
    up = torch.where(some, s["dloss"].double() * T, 0.0)[:, None]
    dX, dW = torch.zeros((N, H), dtype=torch.float64, device=dev), torch.empty((V, H), dtype=torch.float64, device=dev)
    rows = torch.arange(N, device=dev)[:, None].expand_as(at)
    for v0, v1 in blocks:
        w = s["W"][v0:v1].double()
        d = torch.exp(x @ w.T / T - lse[:, None])
        here = ok & (at >= v0) & (at < v1)
        d.index_put_((rows[here], at[here] - v0), -p[here], accumulate=True)
        d *= up
        dX += d @ w
        dW[v0:v1] = d.T @ x
    return {"loss": loss, "lse": lse, "y_top": y_top, "dX": dX, "dW": dW}
