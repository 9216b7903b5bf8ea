"""Layer norm on the GPU against fp64 on the same inputs.

Tolerances, u = 2^-24 and e = half a step of the row type (bf16 2^-8, fp32 u).
A row sum of H <= 65536 terms runs at most 256 deep in a lane and 9 across the
work-group, so a sum is off by at most D u of the sum of its terms' sizes, D =
min(H, 256) + 12.
  mean: D u mean|x|, and one rounding.
  rstd: the mean's error moves the variance by its square, 3 roundings per
    centred square, the sum: relative (D + 6) u, half of that on rstd, and 3
    more; where the row is constant but for rounding the error of the centred
    values, D u |x|, counts beside sqrt(eps).
  Y, dX: products of up to 4 roundings each on terms of their own size, the
    statistics' errors, then e once.
  dgamma, dbeta: at most N / slabs <= N / 512 + 1 terms in a lane, 512 / 4 + 4
    in the fold: D' u of the sum of the terms' sizes."""

import numpy as np
import pytest
import torch

from gpu_common import DEV, B, dev_to_f64, needs_gpu, require_lib

pytestmark = [pytest.mark.gpu, needs_gpu]
U = 2.0 ** -24
TYPES = {"bf16": (torch.bfloat16, 2.0 ** -8), "f32": (torch.float32, U)}


def inputs(N, H, dtype, seed=0, offset=0.3):
    g = torch.Generator().manual_seed(seed)
    dt = TYPES[dtype][0]
    x = (torch.randn(N, H, generator=g) * (0.5 + torch.rand(H, generator=g)) + offset * torch.randn(H, generator=g)).to(dt)
    return x.to(DEV), torch.randn(N, H, generator=g).to(dt).to(DEV), (1 + 0.1 * torch.randn(H, generator=g)).to(DEV), torch.randn(H, generator=g).to(DEV)


def reference(x, gamma, beta, dy, eps):
    x, gamma, dy = (dev_to_f64(t) for t in (x, gamma, dy))
    m = x.mean(1, keepdims=True)
    r = 1 / np.sqrt(((x - m) ** 2).mean(1, keepdims=True) + eps)
    xh = (x - m) * r
    d = dy * gamma
    return dict(m=m, r=r, xh=xh, d=d, dy=dy, x=x, gamma=gamma, Y=xh * gamma + (0 if beta is None else dev_to_f64(beta)),
                dX=r * (d - d.mean(1, keepdims=True) - xh * (d * xh).mean(1, keepdims=True)),
                dgamma=(dy * xh).sum(0), dbeta=dy.sum(0))


def check(x, gamma, beta, dy, dtype, eps=1e-5, name=""):
    N, H = x.shape
    e = TYPES[dtype][1]
    plan = B.lnorm_plan(N, H, B.moe_dtype(x.dtype), eps)
    Y, mean, rstd = B.lnorm_forward(plan, x, gamma, beta)
    dX, dgamma, dbeta = B.lnorm_backward(plan, x, gamma, dy, mean, rstd)
    torch.cuda.synchronize()
    R = reference(x, gamma, beta, dy, eps)
    D = (min(H, 256) + 12) * U
    ax = np.abs(R["x"]).mean(1, keepdims=True)
    m, r = dev_to_f64(mean)[:, None], dev_to_f64(rstd)[:, None]
    m_off = D * ax + U * np.abs(R["m"])
    assert np.all(np.abs(m - R["m"]) <= m_off), (name, "mean")
    # the centred values are off by the mean's error and a rounding of theirs
    c_off = (m_off + U * np.abs(R["x"]).max(1, keepdims=True)) * R["r"]  # in units of 1 / rstd
    r_rel = D + 8 * U + c_off ** 2 + 2 * c_off * np.sqrt((R["xh"] ** 2).mean(1, keepdims=True)) * (1 if H > 1 else 0)
    assert np.all(np.abs(r - R["r"]) <= r_rel * R["r"]), (name, "rstd")
    xh_off = r_rel * np.abs(R["xh"]) + c_off + 3 * U * np.abs(R["xh"])
    g = np.abs(R["gamma"])
    tol = xh_off * g + 4 * U * np.abs(R["xh"] * g) + U * np.abs(R["Y"])
    assert np.all(np.abs(dev_to_f64(Y) - R["Y"]) <= tol * (1 + e) + e * np.abs(R["Y"])), (name, "Y")
    ad, axh = np.abs(R["d"]), np.abs(R["xh"])
    a_off = (D + 4 * U) * ad.mean(1, keepdims=True)
    b_off = (D + 6 * U) * (ad * axh).mean(1, keepdims=True) + (ad * xh_off).mean(1, keepdims=True)
    b = np.abs((R["d"] * R["xh"]).mean(1, keepdims=True))
    inner = ad * 4 * U + a_off + axh * b_off + xh_off * (b + b_off) + 6 * U * (ad + axh * b + np.abs(R["d"].mean(1, keepdims=True)))
    tol = R["r"] * inner * (1 + r_rel) + (r_rel + 2 * U) * np.abs(R["dX"])
    assert np.all(np.abs(dev_to_f64(dX) - R["dX"]) <= tol * (1 + e) + e * np.abs(R["dX"])), (name, "dX")
    Dc = (N / 512 + 1 + 512 / 4 + 8) * U
    ady = np.abs(R["dy"])
    assert np.all(np.abs(dev_to_f64(dgamma) - R["dgamma"]) <= (ady * xh_off).sum(0) + (Dc + 4 * U) * (ady * axh).sum(0)), (name, "dgamma")
    assert np.all(np.abs(dev_to_f64(dbeta) - R["dbeta"]) <= Dc * ady.sum(0)), (name, "dbeta")
    return Y, mean, rstd, dX, dgamma, dbeta


SIZES = [(1, 1), (1, 2048), (3, 7), (777, 1111), (5, 64), (1, 65536), (9, 20000), (600, 512), (33, 7168),
         (257, 1024), (4, 16384), (3, 16392), (130, 2056), (2, 12000), (1025, 72), (7, 4096), (64, 5120), (3000, 256)]


@pytest.mark.parametrize("dtype", sorted(TYPES))
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "%dx%d" % s)
def test_against_oracle(size, dtype):
    require_lib()
    x, dy, gamma, beta = inputs(*size, dtype, seed=size[1])
    check(x, gamma, beta, dy, dtype, name=size)


@pytest.mark.parametrize("dtype", sorted(TYPES))
@pytest.mark.parametrize("H", [129, 768, 2048, 7168])
def test_large_means_constant_rows_and_no_beta(H, dtype):
    require_lib()
    x, dy, gamma, _ = inputs(12, H, dtype, seed=1)
    x = x.clone()
    x[:4] += 1000.0   # a mean far above the spread
    x[4] = 3.25       # a constant row
    x[5] = 0.0
    x[6] = 0.0
    x[6, H // 2] = 100.0
    dy[7] = 0.0
    check(x, gamma, None, dy, dtype, eps=1e-3, name=(H, dtype))


@pytest.mark.parametrize("dtype", sorted(TYPES))
@pytest.mark.parametrize("H", [64, 100, 2048, 4096])
def test_alignment_streams_in_place_and_repeat(H, dtype):
    """Rows that start off a 16-byte step, on another stream, into the middle of
    larger buffers, in place; twice the same bits."""
    require_lib()
    N, dt = 37, TYPES[dtype][0]
    x, dy, gamma, beta = inputs(N, H, dtype, seed=2)
    ref = check(x, gamma, beta, dy, dtype, name="reference")
    again = check(x, gamma, beta, dy, dtype, name="again")
    assert all(torch.equal(a, b) for a, b in zip(ref, again))

    def shifted(t, by=1):
        flat = torch.full((t.numel() + 64,), -7, dtype=t.dtype, device=DEV)
        flat[by:by + t.numel()] = t.reshape(-1)
        return flat[by:by + t.numel()].view(t.shape), flat

    xs, dys, gs, bs = (shifted(t)[0] for t in (x, dy, gamma, beta))
    Y, flat_Y = shifted(torch.zeros_like(x))
    dX, flat_dX = shifted(torch.zeros_like(x))
    plan = B.lnorm_plan(N, H, B.moe_dtype(dt))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    _, mean, rstd = B.lnorm_forward(plan, xs, gs, bs, Y=Y, stream=s)
    B.lnorm_backward(plan, xs, gs, dys, mean, rstd, dX=dX, stream=s)
    s.synchronize()
    e = TYPES[dtype][1]
    for got, want in ((Y, ref[0]), (dX, ref[3])):  # the same sums in another order
        assert np.all(np.abs(dev_to_f64(got) - dev_to_f64(want)) <= 2 * e * np.abs(dev_to_f64(want)) + 1e-5)
    for flat in (flat_Y, flat_dX):
        assert bool((flat[:1] == -7).all()) and bool((flat[1 + N * H:] == -7).all())
    # in place
    x2, dy2 = x.clone(), dy.clone()
    assert torch.equal(B.lnorm_backward(plan, x, gamma, dy2, ref[1], ref[2], dX=dy2)[0], ref[3])
    assert torch.equal(B.lnorm_forward(plan, x2, gamma, beta, Y=x2)[0], ref[0])


def test_gradient_against_differences():
    require_lib()
    N, H = 3, 40
    x, dy, gamma, beta = inputs(N, H, "f32", seed=4)
    plan = B.lnorm_plan(N, H, B.MOE_F32)
    _, mean, rstd = B.lnorm_forward(plan, x, gamma, beta)
    dX, dgamma, dbeta = (dev_to_f64(t) for t in B.lnorm_backward(plan, x, gamma, dy, mean, rstd))
    x64, dy64, g64, b64 = (dev_to_f64(t) for t in (x, dy, gamma, beta))

    def f(x_, g_, b_):
        m = x_.mean(1, keepdims=True)
        return ((x_ - m) / np.sqrt(((x_ - m) ** 2).mean(1, keepdims=True) + 1e-5) * g_ + b_) .ravel() @ dy64.ravel()

    h = 1e-6
    for h_ in range(H):
        e = np.zeros(H)
        e[h_] = h
        assert abs((f(x64, g64 + e, b64) - f(x64, g64 - e, b64)) / (2 * h) - dgamma[h_]) < 1e-4
        assert abs((f(x64, g64, b64 + e) - f(x64, g64, b64 - e)) / (2 * h) - dbeta[h_]) < 1e-4
        for t in range(N):
            q = np.zeros((N, H))
            q[t, h_] = h
            assert abs((f(x64 + q, g64, b64) - f(x64 - q, g64, b64)) / (2 * h) - dX[t, h_]) < 1e-4


def test_no_rows():
    require_lib()
    plan = B.lnorm_plan(0, 100, B.MOE_BF16)
    x = torch.empty((0, 100), dtype=torch.bfloat16, device=DEV)
    gamma, s = torch.ones(100, device=DEV), torch.empty(0, device=DEV)
    B.lnorm_forward(plan, x, gamma)
    _, dg, db = B.lnorm_backward(plan, x, gamma, x, s, s, dgamma=torch.ones(100, device=DEV), dbeta=torch.ones(100, device=DEV))
    assert not dg.any() and not db.any()


@pytest.mark.parametrize("H", [100, 2048])
def test_graph_replays(H):
    require_lib()
    from test_gpu_graph import capture, replay_and_check
    x, dy, gamma, beta = inputs(301, H, "bf16", seed=5)
    plan = B.lnorm_plan(301, H, B.MOE_BF16)
    outs = {"Y": torch.empty_like(x), "mean": torch.empty(301, device=DEV), "rstd": torch.empty(301, device=DEV),
            "dX": torch.empty_like(x), "dgamma": torch.empty(H, device=DEV), "dbeta": torch.empty(H, device=DEV)}
    ws = B.workspace(plan, "bwd", DEV)

    def call():
        B.lnorm_forward(plan, x, gamma, beta, outs["Y"], outs["mean"], outs["rstd"])
        B.lnorm_backward(plan, x, gamma, dy, outs["mean"], outs["rstd"], outs["dX"], outs["dgamma"], outs["dbeta"], ws=ws)

    call()
    torch.cuda.synchronize()
    replay_and_check("lnorm", capture(call), outs, {k: t.clone() for k, t in outs.items()})
