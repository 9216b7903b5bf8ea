"""Distillation over vocabulary strips on the GPU against the fp64 oracle.

Tolerances, u = 2^-24 and e = 2^-8 (half a step of bf16), elementwise:
  a logit: H products summed in fp32, at most (H + 2) u sum |x w| off, dy.
  lse: dy / T, and relative to its sum: 50 u an exponential, 12 u in a slice,
    4 u for each of at most V / 128 steps of the fold; 4 u of its own size.
  p: (80 + 4 R) u relative, R the range of the list's logits over T.
  loss: T^2 times the sum over the list of p's error times |log p - log q|,
    and p times log p's, y's and lse's errors.
  dy: q's relative error (that of lse, of y / T, 50 u), p's, 4 u, times dl; e of
    its size when stored.
  dX, dW: the sum over V (N) terms of dy's error times |w| (|x|), the
    summation V u (N u) of the terms' sizes, and the output's rounding."""

import numpy as np
import pytest
import torch

import oracle
from gpu_common import DEV, B, dev_to_f64, needs_gpu, require_lib

pytestmark = [pytest.mark.gpu, needs_gpu]
U, E = 2.0 ** -24, 2.0 ** -8


class Case:
    def __init__(self, N, H, V, K, seed=0, w_std=0.05):
        r = np.random.default_rng(seed)
        g = torch.Generator().manual_seed(seed)
        self.X = torch.randn(N, H, generator=g).bfloat16().to(DEV)
        self.W = (w_std * torch.randn(V, H, generator=g)).bfloat16().to(DEV)
        self.idx = r.integers(0, V, (N, K)).astype(np.int32)
        self.t = (4 + 2 * r.standard_normal((N, K))).astype(np.float32)
        self.dloss = r.standard_normal(N).astype(np.float32)
        self.N, self.H, self.V, self.K = N, H, V, K


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def run(c, v_chunk, T, dw_dtype=B.MOE_F32, **kw):
    plan = B.kd_plan(c.N, c.H, c.V, v_chunk, c.K, T, dw_dtype=dw_dtype)
    idx, t = dev(c.idx), dev(c.t)
    loss, lse, y_top = B.kd_forward(plan, c.X, c.W, idx, t, **kw)
    dX, dW = B.kd_backward(plan, c.X, c.W, idx, t, lse, y_top, dev(c.dloss), **kw)
    torch.cuda.synchronize()
    return dict(loss=loss, lse=lse, y_top=y_top, dX=dX, dW=dW)


def check(c, v_chunk, T, name=""):
    out = run(c, v_chunk, T)
    got = {k: dev_to_f64(v) for k, v in out.items()}
    X, W = dev_to_f64(c.X), dev_to_f64(c.W)
    loss, lse, y_top = oracle.kd_forward(X, W, c.idx, c.t, T)
    d = oracle.kd_dlogits(X, W, c.idx, c.t, T, c.dloss)
    valid, p, logp = oracle.kd_list(c.idx, c.t, c.V, T)
    size = np.abs(X) @ np.abs(W).T
    dy = (c.H + 2) * U * size
    dy_top = np.where(valid, np.take_along_axis(dy, np.where(valid, c.idx, 0), 1), 0.0)
    assert np.all(np.abs(got["y_top"] - y_top) <= dy_top + U * np.abs(y_top)), (name, "y_top")
    lse_off = dy.max(1) / T + (62 + c.V / 32) * U + 4 * U * np.abs(lse)
    assert np.all(np.abs(got["lse"] - lse) <= lse_off), (name, "lse")
    with np.errstate(invalid="ignore"):
        t = np.where(valid, c.t.astype(np.float64) / T, np.nan)
        R = np.array([np.nanmax(a) - np.nanmin(a) if np.isfinite(a).any() else 0.0 for a in t])
    p_rel = ((80 + 4 * np.minimum(R, 110)) * U)[:, None]
    lp = np.where(valid, logp, 0.0)
    gap = np.where(valid, np.abs(lp - (y_top / T - lse[:, None])), 0.0)
    terms = p * (p_rel * gap + p_rel + dy_top / T + lse_off[:, None] + 8 * U * (np.abs(lp) + np.abs(y_top / T) + np.abs(lse)[:, None]))
    loss_off = T * T * (terms.sum(1) + 10 * U * (p * gap).sum(1)) + 1e-37
    assert np.all(np.abs(got["loss"] - loss) <= loss_off), (name, "loss")
    # the logit gradient's error, entry by entry
    q = np.exp(X @ W.T / T - lse[:, None])
    up = np.where(valid.any(1), np.abs(T * c.dloss.astype(np.float64)), 0.0)[:, None]
    P = np.zeros_like(q)
    rows = np.broadcast_to(np.arange(c.N)[:, None], valid.shape)
    np.add.at(P, (rows[valid], c.idx[valid]), p[valid])
    q_rel = dy / T + lse_off[:, None] + (54 + 2 * np.abs(np.log(np.maximum(q, 1e-30)))) * U
    g_off = up * (q * q_rel + P * (p_rel + c.K * U) + 4 * U * (q + P)) * (1 + E) + E * np.abs(d) + up * 1e-37
    g = np.abs(d) + g_off
    aX, aW = np.abs(X), np.abs(W)
    dX, dW = d @ W, d.T @ X
    tol = g_off @ aW + (c.V + 8) * U * (g @ aW)
    assert np.all(np.abs(got["dX"] - dX) <= tol * (1 + E) + E * np.abs(dX)), (name, "dX")
    tol = g_off.T @ aX + (c.N + 8) * U * (g.T @ aX)
    assert np.all(np.abs(got["dW"] - dW) <= tol + U * np.abs(dW)), (name, "dW")
    empty = ~valid.any(1)
    assert not got["loss"][empty].any() and not got["dX"][empty].any()
    # bf16 dW: the same sums, rounded once
    half = run(c, v_chunk, T, B.MOE_BF16)
    assert torch.equal(half["dW"], out["dW"].bfloat16()) and torch.equal(half["dX"], out["dX"])
    return out


# N, H, V, v_chunk, K, T
SIZES = [(1, 128, 100, 256, 1, 1.0), (300, 256, 257, 256, 4, 2.0), (64, 384, 3000, 512, 64, 0.5),
         (17, 128, 300, 256, 256, 4.0), (5, 128, 1, 256, 2, 1.0), (257, 640, 1000, 1024, 70, 1.0),
         (65, 256, 1300, 512, 9, 1.5), (512, 256, 700, 256, 3, 1.0), (513, 512, 900, 512, 8, 1.0)]


@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
def test_against_oracle(size):
    require_lib()
    N, H, V, v_chunk, K, T = size
    c = Case(N, H, V, K, seed=N)
    # places at the strips' and tiles' edges, an index twice, short and empty lists
    edges = [v for v in (0, 255, 256, 511, 512, V - 1, V // 2) if v < V]
    for i in range(N):
        c.idx[i, i % K] = edges[i % len(edges)]
    if N > 8:
        c.idx[3, 1:] = -1
        c.idx[4] = V
        c.t[5] = -np.inf
        c.t[6, : K // 2] = -np.inf
        c.idx[7] = c.idx[7, 0]
        c.t[8] = np.nan
        c.idx[2, -1] = -2**31
    check(c, v_chunk, T, size)


@pytest.mark.parametrize("T", [1.0, 3.0])
def test_ragged_batch_and_strip_width(T):
    require_lib()
    c = Case(777, 512, 20_000, 16, seed=3)
    short = np.random.default_rng(1).integers(0, 17, 777)
    c.idx[np.arange(16)[None, :] >= short[:, None]] = -1
    out = check(c, 4096, T)
    for vc in (256, 20_224):
        other = run(c, vc, T)
        for k in out:
            assert torch.equal(out[k], other[k]), (vc, k)


@pytest.mark.parametrize("H", [256, 384])
def test_ranges_of_dx_across_strips(H):
    """Several strips, and dX in ranges that start inside a strip and take turns
    on their sums; the same bits for every strip width."""
    require_lib()
    N, V, K, T = 2000, 60_000, 5, 2.0
    c = Case(N, H, V, K, seed=H)
    p = B.kd_plan(N, H, V, 4096, K, T)
    assert p.S > 2
    out = run(c, 4096, T)
    for vc in (256, 1280, 16_640):
        other = run(c, vc, T)
        for k in out:
            assert torch.equal(out[k], other[k]), (vc, k)
    X, W, idx = c.X.double(), c.W.double(), dev(c.idx).long()
    y = X @ W.T / T
    lse = torch.logsumexp(y, 1)
    assert torch.all((out["lse"].double() - lse).abs() <= 2e-5)
    p64 = torch.softmax(dev(c.t).double() / T, 1)
    up = T * dev(c.dloss).double()[:, None]
    g = torch.exp(y - lse[:, None]).scatter_add_(1, idx, -p64) * up
    # e of each gradient (and 1e-4 of it for fp32's share), V u of the sum, e of the result
    dX, dW, aX, aW = g @ W, g.T @ X, X.abs(), W.abs()
    assert torch.all((out["dX"].double() - dX).abs() <= (E + 1e-4 + V * U) * (g.abs() @ aW) + E * dX.abs())
    assert torch.all((out["dW"].double() - dW).abs() <= (E + 1e-4 + N * U) * (g.abs().T @ aX) + U * dW.abs())


def test_extreme_lists():
    require_lib()
    c = Case(40, 128, 500, 8, seed=4)
    c.t[0] = 1e4 * np.arange(8)
    c.t[1] = np.finfo(np.float32).min      # the lowest value is part of the list
    c.t[2, 1:] = np.finfo(np.float32).min
    c.t[3] = np.finfo(np.float32).max
    c.t[4] = 0.0
    c.t[5, :4] = -200.0
    c.dloss[6] = 0.0
    check(c, 256, 1.0)
    check(c, 256, 2.0)


def test_every_list_empty_and_no_tokens():
    require_lib()
    c = Case(33, 128, 300, 3)
    c.idx[:] = -1
    out = run(c, 256, 1.0)
    for k in ("loss", "y_top", "dX", "dW"):
        assert not out[k].any(), k
    c = Case(0, 128, 300, 3)
    for dt in (B.MOE_F32, B.MOE_BF16):
        assert not run(c, 256, 1.0, dt)["dW"].any()


def test_other_stream_and_untouched_neighbours():
    require_lib()
    c = Case(65, 128, 700, 5, seed=8)
    ref = run(c, 256, 2.0, B.MOE_BF16)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = run(c, 256, 2.0, B.MOE_BF16, stream=s)
    for k in ref:
        assert torch.equal(ref[k], got[k]), k
    whole = {k: torch.full((v.shape[0] + 2, *v.shape[1:]), -7, dtype=v.dtype, device=DEV) for k, v in ref.items()}
    plan = B.kd_plan(65, 128, 700, 256, 5, 2.0, dw_dtype=B.MOE_BF16)
    o = {k: v[1:-1] for k, v in whole.items()}
    B.kd_forward(plan, c.X, c.W, dev(c.idx), dev(c.t), o["loss"], o["lse"], o["y_top"])
    B.kd_backward(plan, c.X, c.W, dev(c.idx), dev(c.t), o["lse"], o["y_top"], dev(c.dloss), o["dX"], o["dW"])
    for k in ref:
        assert torch.equal(o[k], ref[k]), k
        assert bool((whole[k][0] == -7).all()) and bool((whole[k][-1] == -7).all()), k


def test_full_size_sampled():
    """The vocabulary workload's sizes, on sampled tokens and vocabulary rows."""
    require_lib()
    N, H, V, K, T = 8192, 7168, 200_000, 32, 1.0
    g = torch.Generator(device=DEV).manual_seed(0)
    X = torch.randn(N, H, generator=g, device=DEV).bfloat16()
    W = (0.02 * torch.randn(V, H, generator=g, device=DEV)).bfloat16()
    idx = torch.randint(0, V, (N, K), generator=g, device=DEV, dtype=torch.int32)
    t = 8 + 2 * torch.randn(N, K, generator=g, device=DEV)
    dloss = torch.full((N,), 1.0 / N, device=DEV)
    plan = B.kd_plan(N, H, V, 8192, K, T, dw_dtype=B.MOE_BF16)
    loss, lse, y_top = B.kd_forward(plan, X, W, idx, t)
    dX, dW = B.kd_backward(plan, X, W, idx, t, lse, y_top, dloss)
    rows = torch.tensor([0, 1, 255, 256, 4095, 8190, 8191], device=DEV)
    y = X[rows].double() @ W.double().T  # 7 rows of logits
    ref_lse = torch.logsumexp(y, 1)
    assert torch.all((lse[rows].double() - ref_lse).abs() <= 2e-5)
    at = idx[rows].long()
    assert torch.all((y_top[rows].double() - y.gather(1, at)).abs() <= 2e-5)
    p = torch.softmax(t[rows].double(), 1)
    ref = (p * (p.log() - y.gather(1, at) + ref_lse[:, None])).sum(1)
    assert torch.all((loss[rows].double() - ref).abs() <= 1e-5 * ref.abs() + 2e-5)
    d = torch.exp(y - ref_lse[:, None]).scatter_add_(1, at, -p) / N
    dx = d @ W.double()
    assert torch.all((dX[rows].double() - dx).abs() <= E * dx.abs() + 1.01 * E * (d.abs() @ W.double().abs()))
    # the rows of W that the first sampled token's list names
    for v in at[0, :4].tolist() + [V - 1]:
        q = torch.exp(X.double() @ W[v].double() - lse.double())
        q -= torch.where(idx == v, torch.softmax(t.double(), 1), 0.0).sum(1)
        ref = (q / N) @ X.double()
        tol = (1.05 * E * q.abs() / N) @ X.double().abs() + E * ref.abs()
        assert torch.all((dW[v].double() - ref).abs() <= tol)


def test_graph_replays():
    require_lib()
    from test_gpu_graph import capture, replay_and_check
    c = Case(300, 256, 3000, 9, seed=2)
    ref = run(c, 1024, 2.0)
    outs = {k: torch.empty_like(v) for k, v in ref.items()}
    plan = B.kd_plan(300, 256, 3000, 1024, 9, 2.0)
    ws, idx, t, dl = B.workspace(plan, "both", DEV), dev(c.idx), dev(c.t), dev(c.dloss)

    def call():
        B.kd_forward(plan, c.X, c.W, idx, t, outs["loss"], outs["lse"], outs["y_top"], ws=ws)
        B.kd_backward(plan, c.X, c.W, idx, t, outs["lse"], outs["y_top"], dl, outs["dX"], outs["dW"], ws=ws)

    replay_and_check("distill", capture(call), outs, ref)


@pytest.mark.parametrize("T", [0.5, 0.25, 0.3])
def test_finite_logits_whose_quotients_overflow(T):
    """An entry is part of the list by its logit, not by logit / T; the softmax
    is of the differences."""
    require_lib()
    c = Case(40, 128, 500, 8, seed=5)
    lo, hi = np.finfo(np.float32).min, np.finfo(np.float32).max
    c.t[0] = lo                # all equal, each 1 / 8
    c.t[1] = hi
    c.t[2, 1:] = lo            # one real entry beside the lowest value
    c.t[3, ::2] = lo
    c.t[4, ::2] = hi
    c.t[5] = [hi, lo] * 4
    c.t[6, :3] = -np.inf
    c.t[6, 3:] = lo
    c.t[7] = np.nan
    c.t[8] = hi * (1 - 2.0 ** -20 * np.arange(8))
    out = check(c, 256, T)
    assert not out["loss"][7] and bool((out["loss"][:7] > 0).all())


# N, H, V, v_chunk, K, T: 128 x 256 logit tiles in both passes, ragged in rows and columns
FEW = [(100, 640, 40_001, 1024, 5, 1.0), (129, 768, 22_100, 256, 9, 2.0), (65, 1024, 33_000, 4096, 70, 1.0)]


@pytest.mark.parametrize("size", FEW, ids=lambda s: "x".join(map(str, s)))
def test_long_rows_of_few_tokens(size):
    require_lib()
    N, H, V, v_chunk, K, T = size
    c = Case(N, H, V, K, seed=H, w_std=0.02)
    c.idx[:, 0] = [(V - 1, 0, 255, 256, V - V % 256, V - V % 256 - 1)[i % 6] for i in range(N)]
    c.idx[5] = -1
    c.idx[N - 1, 1:] = c.idx[N - 1, 0]
    check(c, v_chunk, T, size)


# N, H, V, and widths for which the strips differ; of the second, dX is one sum
WIDTHS = [(777, 512, 60_000, (4096, 256, 20_224)), (8200, 640, 10_001, (1024, 4096, 2048))]


@pytest.mark.parametrize("size", WIDTHS, ids=lambda s: "x".join(map(str, s[:3])))
def test_same_bits_for_strips_that_differ(size):
    require_lib()
    N, H, V, widths = size
    K, T = 6, 2.0
    strips = [B.kd_plan(N, H, V, vc, K, T).strip for vc in widths]
    assert len(set(strips)) == len(widths) and all(s < V and V % s for s in strips), strips
    c = Case(N, H, V, K, seed=H, w_std=0.03)
    c.idx[:6, 0] = [v - d for v in strips for d in (0, 1)]  # either side of the first edges
    c.idx[9] = -1
    out = run(c, widths[0], T)
    for vc in widths[1:]:
        other = run(c, vc, T)
        for k in out:
            assert torch.equal(out[k], other[k]), (vc, k)
    half = run(c, widths[1], T, B.MOE_BF16)
    assert torch.equal(half["dW"], out["dW"].bfloat16()) and torch.equal(half["dX"], out["dX"])
    X, W, idx = c.X.double(), c.W.double(), dev(c.idx).long()
    y = X @ W.T / T
    lse = torch.logsumexp(y, 1)
    # y's sum of H products, the exponentials' and the fold's roundings, at most
    assert torch.all((out["lse"].double() - lse).abs() <= (H + 2) * U * (X.abs() @ W.abs().T).amax(1) / T + (62 + V / 32) * U + 4 * U * lse.abs())
    ok = idx >= 0
    p64 = torch.where(ok, torch.softmax(dev(c.t).double() / T, 1), 0.0)
    up = torch.where(ok.any(1), T * dev(c.dloss).double(), 0.0)[:, None]
    g = torch.exp(y - lse[:, None]).scatter_add_(1, idx.clamp_min(0), -p64) * up
    # e of each gradient (and 1e-4 of it for fp32's share), V u (N u) of the sum, e (u) of the result
    dX, dW, aX, aW = g @ W, g.T @ X, X.abs(), W.abs()
    assert torch.all((out["dX"].double() - dX).abs() <= (E + 1e-4 + V * U) * (g.abs() @ aW) + E * dX.abs())
    assert torch.all((out["dW"].double() - dW).abs() <= (E + 1e-4 + N * U) * (g.abs().T @ aX) + U * dW.abs())
    assert not out["dX"][9].any() and not out["loss"][9]
