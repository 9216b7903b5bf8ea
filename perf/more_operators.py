"""Cases of the 8-bit path of an expert layer and the operators along it: root-mean-square norm with the residual's
addition, products grouped by expert in bfloat16 and in 8 bits, and SwiGLU whose activation checkpoints have 8 bits.
`run` computes a case in plain torch operations, or, where `own` is true, with the library's kernels.

Rows in 8 bits are e4m3 numbers, padded with zeros to a multiple of 128, with a power of two for each row and 128
columns as its scale (E8M0 bytes, four to a step): the smallest, from 2^-110 up, under which the block's largest
magnitude is at most 448.  Weights have one scale for each 128 x 128.  `run` returns the values that they stand for."""

import math

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
E4M3, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu


# ---- cases


def _rms(name, N, H, dtype, residual, out8, way):
    return {"name": name, "op": "rms", "N": N, "H": H, "dtype": dtype, "residual": residual, "out8": out8, "way": way}


def _act8(name, N, F, dtype, way):
    return {"name": name, "op": "act8", "N": N, "F": F, "dtype": dtype, "way": way}


def _gmm(name, R, K, N, E, skew, way):
    return {"name": name, "op": "gmm", "R": R, "K": K, "N": N, "E": E, "skew": skew, "way": way}


def _gmm8(name, R, K, N, E, skew, way):
    return {"name": name, "op": "gmm8", "R": R, "K": K, "N": N, "E": E, "skew": skew, "way": way}


def listed():
    return [
        # one token's hidden row onto the residual stream and into 8 bits; latency is all there is
        _rms("rms_one_token", 1, 2048, "bf16", True, True, "fwd"),
        # the 65,536-token training batch, forward into 8 bits and backward
        _rms("rms_train", 65536, 2048, "bf16", True, True, "both"),
        # a ragged batch of rows that no vector width divides, in 32 bits, without residual
        _rms("rms_odd_f32", 777, 1111, "f32", False, False, "both"),
        # the expert activations of 16,384 tokens with 8 experts each, forward and backward
        _act8("act8_train", 131072, 1536, "bf16", "both"),
        # a short ragged batch from products in 32 bits
        _act8("act8_odd_f32", 779, 1000, "f32", "both"),
        # 16 tokens of a served model with 8 of 64 experts each: the weights' bytes are all there is
        _gmm("gmm_decode", 128, 2048, 1408, 64, 0.0, "fwd"),
        # 4096 tokens with 8 of 64 experts each: forward, and both gradients
        _gmm("gmm_train", 32768, 2048, 1408, 64, 0.2, "all"),
        # few rows of odd sizes over experts of which some have none
        _gmm("gmm_ragged", 1000, 520, 264, 7, 1.5, "all"),
        # one token through a dense projection in 8 bits
        _gmm8("gmm8_one_token", 1, 7168, 2048, 1, 0.0, "fwd"),
        # the same projection for a batch of 8192 tokens
        _gmm8("gmm8_dense", 8192, 7168, 2048, 1, 0.0, "fwd"),
        # 16,384 tokens with 8 of 128 experts each, some experts much hotter than others
        _gmm8("gmm8_experts", 131072, 4096, 1536, 128, 0.5, "fwd"),
        # the weight gradients of 4096 tokens' products, from rows kept in 8 bits
        _gmm8("gmm8_dw", 32768, 2048, 1408, 64, 0.2, "dw"),
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["rms", "act8", "gmm", "gmm8"])
    if op == "rms":
        N, H = _spread(rng, 1, 65536), _spread(rng, 64, 12000)
        if rng.random() < 0.7:
            H = -(-H // 64) * 64
        c = _rms("", max(1, min(N, 134_217_728 // H)), H, rng.choice(["bf16", "bf16", "f32"]), rng.random() < 0.6, rng.random() < 0.6,
                 rng.choice(["fwd", "bwd", "both"]))
    elif op == "act8":
        N, F = _spread(rng, 1, 131072), _spread(rng, 32, 8192)
        if rng.random() < 0.7:
            F = -(-F // 64) * 64
        dt = rng.choice(["bf16", "bf16", "f32"])
        c = _act8("", max(1, min(N, 100_000_000 // F)), F, dt, rng.choice(["fwd", "both"]))
    else:
        R, E = _spread(rng, 1, 32768), _spread(rng, 1, 128)
        K, N = 8 * _spread(rng, 8, 896), 8 * _spread(rng, 8, 512)
        if op == "gmm8" and rng.random() < 0.3:
            K -= rng.randint(1, 7)  # the rows' padding takes any width
        E = max(1, min(E, 400_000_000 // (K * N)))
        R = max(1, min(R, 280_000_000_000 // (2 * K * N)))
        skew = rng.choice([0.0, 0.2, 0.5, 1.0])
        c = _gmm("", R, K, N, E, skew, rng.choice(["fwd", "all"])) if op == "gmm" else _gmm8("", R, K, N, E, skew, rng.choice(["fwd", "fwd", "dw"]))
    del c["name"]
    return c


# ---- 8-bit rows: what they are, in plain operations


def _exponent(amax):
    """The scale's exponent for a block's largest magnitude: amax = m 2^x with 0.5 <= m < 1, and 448 = 0.875 2^9."""
    m, x = torch.frexp(amax)
    return torch.where(amax > 0, x - 9 + (m > 0.875), -110).clamp_(-110, 127)


def _quantise(x):
    """Rows x [R][W], W a multiple of 128, as (e4m3 numbers, exponents [R][W / 128])."""
    v = x.view(x.shape[0], -1, 128)
    big = torch.where(torch.isfinite(v), v.abs(), 0.0).amax(2)
    e = _exponent(big)
    scaled = torch.ldexp(v, -e[:, :, None])  # e and -e both have a power of two in 32 bits
    return scaled.to(E4M3).view(x.shape), e


def _padded(x):
    return torch.nn.functional.pad(x, (0, -x.shape[1] % 128))


def _values(q, e):
    return torch.ldexp(q.float().view(q.shape[0], -1, 128), e[:, :, None]).view(q.shape)


def _through8(x):
    """The values (bfloat16 holds each) that the rows x [N][H] have in 8 bits."""
    return _values(*_quantise(_padded(x)))[:, :x.shape[1]].to(torch.bfloat16)


def _scale_bytes(e):
    """Exponents [R][B] as E8M0 bytes in rows of a multiple of four, the rest 2^0."""
    return torch.nn.functional.pad((e + 127).to(torch.uint8), (0, -e.shape[1] % 4), value=127).contiguous().view(E8M0)


def _exponents(s, width):
    return s.view(torch.uint8)[..., :-(-width // 128)].int() - 127


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

    if c["op"] == "rms":
        N, H, dt = c["N"], c["H"], DTYPES[c["dtype"]]
        # hidden rows: channels with widths of their own, a few far wider than the rest
        wide = 0.5 + torch.rand(H, generator=g, device=DEV)
        wide[torch.rand(H, generator=g, device=DEV) < 0.01] *= 8
        s["X"] = (normal(N, H) * wide).to(dt)
        s["residual"] = normal(N, H, std=2.0, dtype=dt) if c["residual"] and c["way"] != "bwd" else None
        s["gamma"], s["eps"] = 1 + normal(H, std=0.1), 1e-6
        if c["way"] != "fwd":
            s["dY"] = normal(N, H, dtype=dt)
            s["dS"] = normal(N, H, dtype=dt) if c["residual"] else None
        if c["way"] == "bwd":  # what the forward pass has kept
            s["rstd"] = (s["X"].double().square().mean(1) + s["eps"]).rsqrt().float()
        if own:
            from memory_bounded_expert_amd import binding as B
            s["plan"] = B.rms_plan(N, H, B.moe_dtype(dt), s["eps"])
            s["ws"] = B.workspace(s["plan"], "bwd", torch.device("cuda:0")) if c["way"] != "fwd" else None
            s["plan8"] = B.q8_plan(N, H, B.MOE_BF16)
    elif c["op"] == "act8":
        N, F, dt = c["N"], c["F"], DTYPES[c["dtype"]]
        s["A"], s["U"] = normal(N, F, std=1.5, dtype=dt), normal(N, F, dtype=dt)
        s["dH"] = normal(N, F, dtype=dt) if c["way"] == "both" else None
        if own:
            from memory_bounded_expert_amd import binding as B
            s["plan"], s["plan8"] = B.q8_plan(N, F, B.moe_dtype(dt)), B.q8_plan(N, F, B.MOE_BF16)
    else:
        R, K, N, E = c["R"], c["K"], c["N"], c["E"]
        # rows of each expert: shares r^-skew in an order of their own, drawn
        host = torch.Generator()
        host.manual_seed(seed)
        share = torch.arange(1, E + 1, dtype=torch.float64).pow(-c["skew"])[torch.randperm(E, generator=host)]
        to = torch.multinomial(share, R, replacement=True, generator=host)
        sizes = torch.bincount(to, minlength=E)
        s["cap"] = int(sizes.max())
        s["offsets"] = torch.nn.functional.pad(sizes.cumsum(0), (1, 0)).int().to(DEV)
        s["X"] = normal(R, K, dtype=torch.bfloat16)
        if c["op"] == "gmm":
            s["W"] = normal(E, K, N, std=0.02, dtype=torch.bfloat16)
        else:
            q, e = _quantise(_padded(s.pop("X").float()))
            s["Xq"], s["Xs"] = q, _scale_bytes(e)
        if c["op"] == "gmm8" and c["way"] == "fwd":
            # weights, an expert at a time; their last blocks are short where 128 does not divide N or K
            kp, nb = -(-K // 128) * 128, -(-N // 128)
            s["Wq"] = torch.empty((E, N, kp), dtype=E4M3, device=DEV)
            s["Ws"] = torch.empty((E, nb, -(-kp // 512) * 4), dtype=E8M0, device=DEV)
            for i in range(E):
                w = torch.zeros((nb * 128, kp), device=DEV)
                w[:N, :K] = torch.randn((N, K), generator=g, device=DEV) * (0.01 + 0.02 * torch.rand((N, 1), generator=g, device=DEV))
                e = _exponent(w.view(nb, 128, kp // 128, 128).abs().amax((1, 3)))
                full = e.repeat_interleave(128, 0).repeat_interleave(128, 1)
                s["Wq"][i] = torch.ldexp(w, -full)[:N].to(E4M3)
                s["Ws"][i] = _scale_bytes(e)
        if c["way"] in ("all", "dw"):
            s["dY"] = normal(R, N, dtype=torch.bfloat16)
        if own:
            from memory_bounded_expert_amd import binding as B
            s["plan"] = B.gmm_plan(R, K, N, E, B.GMM_BF16 if c["op"] == "gmm" else B.GMM_Q8)
            s["ws"] = B.workspace(s["plan"], "both", torch.device("cuda:0"))
    return s


# ---- one pass


def run(s):
    return {"rms": _run_rms, "act8": _run_act8, "gmm": _run_gmm, "gmm8": _run_gmm8}[s["case"]["op"]](s)


def _run_rms(s):
    c, out = s["case"], {}
    if own:
        from memory_bounded_expert_amd import binding as B
        S, rstd = s["X"], s.get("rstd")
        if c["way"] != "bwd":
            if c["out8"]:
                q, sc, S, rstd = B.rms_forward_q8(s["plan"], s["X"], s["gamma"], s["residual"])
                out["Y"] = B.q8_unpack(s["plan8"], q, sc)
            else:
                out["Y"], S, rstd = B.rms_forward(s["plan"], s["X"], s["gamma"], s["residual"])
            out["S"], out["rstd"] = S, rstd
        if c["way"] != "fwd":
            out["dX"], out["dgamma"] = B.rms_backward(s["plan"], S, s["gamma"], s["dY"], rstd, s["dS"], ws=s["ws"])
        return out
    dt = s["X"].dtype
    S = s["X"] if s["residual"] is None else (s["X"].float() + s["residual"].float()).to(dt)
    x = S.float()
    if c["way"] == "bwd":
        rstd = s["rstd"]
    else:
        rstd = (x.square().mean(1) + s["eps"]).rsqrt()
        y = x * rstd[:, None] * s["gamma"]
        out["Y"] = _through8(y) if c["out8"] else y.to(dt)
        out["S"], out["rstd"] = S, rstd
    if c["way"] != "fwd":
        dy, xh = s["dY"].float(), x * rstd[:, None]
        d = dy * s["gamma"]
        dx = rstd[:, None] * (d - xh * (d * xh).mean(1, keepdim=True))
        if s["dS"] is not None:
            dx = dx + s["dS"].float()
        out["dX"], out["dgamma"] = dx.to(dt), (dy * xh).sum(0)
    return out


def _run_act8(s):
    c = s["case"]
    if own:
        from memory_bounded_expert_amd import binding as B
        hq, hs, kept = B.q8_swiglu_forward(s["plan"], s["A"], s["U"])
        out = {"H": B.q8_unpack(s["plan8"], hq, hs)}
        if c["way"] == "both":
            out["dA"], out["dU"] = B.q8_swiglu_backward(s["plan"], kept, s["dH"])
        else:
            out["A"], out["U"] = B.q8_unpack(s["plan8"], *kept[:2]), B.q8_unpack(s["plan8"], *kept[2:])
        return out
    a, u = s["A"].float(), s["U"].float()
    out = {"H": _through8(a / (1 + torch.exp(-a)) * u)}
    a8, u8 = _through8(a), _through8(u)
    if c["way"] == "both":
        a, u, dh = a8.float(), u8.float(), s["dH"].float()
        gate = 1 / (1 + torch.exp(-a))
        out["dA"] = (dh * u * gate * (1 + a * (1 - gate))).to(s["A"].dtype)
        out["dU"] = (dh * a * gate).to(s["A"].dtype)
    else:
        out["A"], out["U"] = a8, u8
    return out


def _by_expert(s, rows, of, at):
    """Rows [R][W] as [E][cap][W] in 32 bits, the places that no row has 0."""
    out = torch.zeros((s["case"]["E"], s["cap"], rows.shape[1]), device=DEV)
    out[of, at] = rows
    return out


def _places(s):
    row = torch.arange(s["case"]["R"], device=DEV)
    of = torch.searchsorted(s["offsets"][1:], row, right=True)
    return of, row - s["offsets"][of]


def _run_gmm(s):
    c, X, W, off = s["case"], s["X"], s["W"], s["offsets"]
    if own:
        from memory_bounded_expert_amd import binding as B
        out = {"Y": B.gmm_forward(s["plan"], X, W, off, ws=s["ws"])}
        if c["way"] == "all":
            out["dX"] = B.gmm_backward_dx(s["plan"], s["dY"], W, off, ws=s["ws"])
            out["dW"] = B.gmm_backward_dw(s["plan"], X, s["dY"], off, ws=s["ws"])
        return out
    of, at = _places(s)
    x, w = _by_expert(s, X.float(), of, at), W.float()
    out = {"Y": torch.bmm(x, w)[of, at].to(torch.bfloat16)}
    if c["way"] == "all":
        d = _by_expert(s, s["dY"].float(), of, at)
        out["dX"] = torch.bmm(d, w.transpose(1, 2))[of, at].to(torch.bfloat16)
        out["dW"] = torch.bmm(x.transpose(1, 2), d)
    return out


def _run_gmm8(s):
    c, off = s["case"], s["offsets"]
    K, N = c["K"], c["N"]
    if own:
        from memory_bounded_expert_amd import binding as B
        if c["way"] == "dw":
            return {"dW": B.gmm8_backward_dw(s["plan"], s["Xq"], s["Xs"], s["dY"], off, ws=s["ws"])}
        return {"Y": B.gmm8_forward(s["plan"], s["Xq"], s["Xs"], s["Wq"], s["Ws"], off, ws=s["ws"])}
    of, at = _places(s)
    x = _by_expert(s, _values(s["Xq"], _exponents(s["Xs"], K))[:, :K], of, at)
    if c["way"] == "dw":
        return {"dW": torch.bmm(x.transpose(1, 2), _by_expert(s, s["dY"].float(), of, at))}
    e = _exponents(s["Ws"], K).repeat_interleave(128, 1)[:, :N]
    w = _values(s["Wq"].view(c["E"] * N, -1), e.reshape(c["E"] * N, -1)).view(c["E"], N, -1)[:, :, :K]
    return {"Y": torch.bmm(x, w.transpose(1, 2))[of, at].to(torch.bfloat16)}


# ---- what a pass cannot do without


def work(case):
    c = case
    if c["op"] == "rms":
        N, H, b = c["N"], c["H"], 2 if c["dtype"] == "bf16" else 4
        rows = 0.0
        if c["way"] != "bwd":
            rows += b + (2 * b if c["residual"] else 0) + (1 + 1 / 128 if c["out8"] else b)
        if c["way"] != "fwd":
            rows += (2 if c["way"] == "both" else 3) * b + (b if c["residual"] else 0)
        return {"bytes": int(N * H * rows) + 4 * N + 8 * H, "flops": N * H * {"fwd": 6, "bwd": 10, "both": 16}[c["way"]]}
    if c["op"] == "act8":
        b = 2 if c["dtype"] == "bf16" else 4
        each = 2 * b + 3 * (1 + 1 / 128) + (3 * b if c["way"] == "both" else 0)
        return {"bytes": int(c["N"] * c["F"] * each), "flops": c["N"] * c["F"] * (20 if c["way"] == "both" else 10)}
    R, K, N, E = c["R"], c["K"], c["N"], c["E"]
    share = [(r + 1) ** -c["skew"] for r in range(E)]
    seen = sum(1 - (1 - p / sum(share)) ** R for p in share)  # experts that have rows
    if c["op"] == "gmm":
        moved = R * K * 2 + int(seen) * K * N * 2 + R * N * 2
        if c["way"] == "all":
            moved += R * N * 2 + R * K * 2 + E * K * N * 4
        return {"bytes": moved, "flops": 2 * R * K * N * (3 if c["way"] == "all" else 1)}
    if c["way"] == "dw":
        return {"bytes": R * K + R * N * 2 + E * K * N * 4, "flops": 2 * R * K * N}
    return {"bytes": R * K + int(seen) * K * N + R * N * 2, "flops": 2 * R * K * N}


# ---- the definitions in 64 bits


def exact(case, seed):
    c, s = dict(case), prepare(case, seed)
    return {"rms": _exact_rms, "act8": _exact_act8, "gmm": _exact_gmm, "gmm8": _exact_gmm8}[c["op"]](c, s)


def _nearest8(x):
    """The values that rows x [N][H] in 64 bits have in 8 bits, block by block of columns: the nearest multiple of
    each value's step, ties to the even one."""
    parts = []
    for h in range(0, x.shape[1], 128):
        v = x[:, h:h + 128]
        top = v.abs().amax(1, keepdim=True)
        e = torch.ceil(torch.log2(top / 448)).clamp_min_(-110)
        e = torch.where(top * torch.exp2(-e) > 448, e + 1, e)  # the logarithm's own rounding
        e = torch.where((top * torch.exp2(1 - e) <= 448) & (e > -110), e - 1, e)
        y = v * torch.exp2(-e)
        step = torch.exp2(torch.frexp(y)[1].clamp_min(-5).double() - 4)  # three bits after the leading one; 2^-9 at least
        parts.append(torch.round(y / step) * step * torch.exp2(e))
    return torch.cat(parts, 1)


def _exact_rms(c, s):
    out, x = {}, s["X"].double()
    if s["residual"] is not None:
        x = (x + s["residual"].double()).to(s["X"].dtype).double()
    if c["way"] == "bwd":
        r = s["rstd"].double()
    else:
        r = 1 / torch.sqrt(torch.linalg.vector_norm(x, dim=1) ** 2 / c["H"] + s["eps"])
        y = torch.einsum("nh,n,h->nh", x, r, s["gamma"].double())
        out["Y"] = _nearest8(y) if c["out8"] else y
        out["S"], out["rstd"] = x, r
    if c["way"] != "fwd":
        dy, gamma = s["dY"].double(), s["gamma"].double()
        along = ((dy * x) @ gamma) * r ** 3 / c["H"]
        out["dX"] = torch.addcmul(-along[:, None] * x, dy * r[:, None], gamma)
        if s["dS"] is not None:
            out["dX"] += s["dS"].double()
        out["dgamma"] = r @ (dy * x)
    return out


def _exact_act8(c, s):
    a, u = s["A"].double(), s["U"].double()
    out = {"H": _nearest8(torch.nn.functional.silu(a) * u)}
    a, u = _nearest8(a), _nearest8(u)
    if c["way"] == "fwd":
        return dict(out, A=a, U=u)
    dh, sg = s["dH"].double(), torch.sigmoid(a)
    out["dA"] = dh * u * (sg + a * sg * torch.sigmoid(-a))
    out["dU"] = dh * torch.nn.functional.silu(a)
    return out


def _exact_gmm(c, s):
    ends = s["offsets"].tolist()
    out = {"Y": torch.empty((c["R"], c["N"]), dtype=torch.float64, device=DEV)}
    if c["way"] == "all":
        out["dX"] = torch.empty((c["R"], c["K"]), dtype=torch.float64, device=DEV)
        out["dW"] = torch.empty((c["E"], c["K"], c["N"]), dtype=torch.float64, device=DEV)
    for e in range(c["E"]):
        rows = slice(ends[e], ends[e + 1])
        x, w = s["X"][rows].double(), s["W"][e].double()
        out["Y"][rows] = x @ w
        if c["way"] == "all":
            d = s["dY"][rows].double()
            out["dX"][rows] = d @ w.T.contiguous()
            out["dW"][e] = x.T.contiguous() @ d
    return out


def _exact_gmm8(c, s):
    ends, K, N = s["offsets"].tolist(), c["K"], c["N"]

    def powers(sc, rows):
        p = torch.exp2(sc.view(torch.uint8).double() - 127)
        return p.repeat_interleave(128, 1)[:, :K].repeat_interleave(rows, 0)

    first = c["way"] == "fwd"
    out = torch.empty((c["R"], N) if first else (c["E"], K, N), dtype=torch.float64, device=DEV)
    for e in range(c["E"]):
        rows = slice(ends[e], ends[e + 1])
        x = s["Xq"][rows].to(torch.float64)[:, :K] * powers(s["Xs"][rows], 1)
        if first:
            w = s["Wq"][e].to(torch.float64)[:, :K] * powers(s["Ws"][e], 128)[:N]
            out[rows] = x @ w.T.contiguous()
        else:
            out[e] = x.T.contiguous() @ s["dY"][rows].double()
    return {"Y" if first else "dW": out}
