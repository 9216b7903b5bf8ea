"""Routing by scores on the GPU against the fp64 oracle, and the layer under a
given routing.

topk_idx has to equal the oracle's on every input.  Tolerances, in units of
u = 2^-24 (half a step of fp32): a gate is made of at most two exponentials
(2 u each, plus 2 u per unit of their arguments' range R, the argument being
rounded before and scaled inside), two sums of positive terms (at most 22
roundings each: 16 in a lane, 6 across the wave) and up to four further
roundings of at most 2 u, so (64 + 4 R) u relative bounds it.  A gradient is w (scale
dg - dot) (1 - s), with w as a gate and dot a sum of k <= 64 products: each of
the two terms is off by at most (128 + 8 R) u of its own size."""

import numpy as np
import pytest
import torch

import datagen
import oracle
from gpu_common import DEV, B, DevInputs, dev_to_f64, needs_gpu, plan_for, require_lib, say

pytestmark = [pytest.mark.gpu, needs_gpu]
U = 2.0 ** -24

# N, E, k, groups, kept, group_top
SHAPES = [
    (1, 1, 1, 1, 1, 1), (1, 256, 8, 8, 4, 2), (5, 60, 7, 4, 2, 2), (3, 8, 8, 1, 1, 1),
    (64, 64, 64, 1, 1, 1), (333, 256, 8, 8, 4, 2), (130, 1000, 32, 8, 3, 2),
    (77, 1024, 64, 64, 16, 2), (257, 896, 16, 1, 1, 1), (100, 72, 3, 24, 5, 1),
    (50, 16, 3, 16, 4, 2), (1001, 128, 8, 1, 1, 1), (19, 320, 5, 2, 1, 2), (21, 513, 4, 3, 2, 2),
    (37, 260, 17, 1, 1, 1), (90, 250, 32, 1, 1, 1), (33, 100, 40, 1, 1, 1), (41, 40, 33, 1, 1, 1),
    (29, 256, 48, 8, 4, 2), (23, 192, 64, 6, 3, 2), (31, 128, 16, 1, 1, 1), (35, 128, 17, 1, 1, 1),
]


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def check(l, bias, up, k, score, g, kept, top, renorm, scale, name=""):
    l = np.asarray(l, np.float32)
    N, E = l.shape
    plan = B.route_plan(N, E, k, score, g, kept, top, renorm, scale)
    dl = dev(l)
    idx, gates = B.route_forward(plan, dl, None if bias is None else dev(bias))
    grad = B.route_backward(plan, dl, idx, dev(up))
    torch.cuda.synchronize()
    want = oracle.route_select(l, k, score, bias, g, kept, top)
    got = idx.cpu().numpy().astype(np.int64)
    assert np.array_equal(got, want), (name, np.nonzero((got != want).any(1))[0][:5])
    ref = oracle.route_gates(l, want, score, renorm, scale)
    fin = np.where(np.isfinite(l), l, np.nan)
    with np.errstate(invalid="ignore"):
        import warnings
        with warnings.catch_warnings():
            warnings.simplefilter("ignore")
            R = np.nan_to_num(np.nanmax(fin, 1) - np.nanmin(fin, 1)) + np.nan_to_num(np.nanmax(np.abs(fin), 1))
    R = np.minimum(R, 110.0)[:, None]  # exponentials past that are 0
    # below the smallest normal number a gate keeps an absolute step only
    assert np.all(np.abs(dev_to_f64(gates) - ref) <= (64 + 4 * R) * U * ref + 2e-38 * scale), name
    s = np.exp(oracle.route_log_scores(l, score))
    tol = np.zeros((N, E))
    # the two terms' sizes per expert
    dot = (ref * np.abs(up)).sum(1, keepdims=True)
    one = np.zeros((N, E))
    np.add.at(one, (np.arange(N)[:, None], want), ref * np.abs(up) + (ref / scale * dot if renorm else 0))
    tol = one + (s * dot if score == "softmax" and not renorm else 0)
    ref_d = oracle.route_backward(l, want, up, score, renorm, scale)
    err = np.abs(dev_to_f64(grad) - ref_d)
    assert np.all(err <= (128 + 8 * R) * U * tol + 4e-38 * scale), (name, err.max())
    return idx, gates, grad


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_against_oracle(shape, score):
    require_lib()
    N, E, k, g, kept, top = shape
    rng = np.random.default_rng(E + k)
    l = (1.5 * rng.standard_normal((N, E))).astype(np.float32)
    up = rng.standard_normal((N, k)).astype(np.float32)
    bias = (0.1 * rng.standard_normal(E)).astype(np.float32)
    for b in (None, bias):
        for renorm, scale in ((True, 1.0), (False, 2.5)):
            check(l, b, up, k, score, g, kept, top, renorm, scale, (shape, score, b is None, renorm))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups", [(1, 1), (8, 3)])
def test_masks_ties_and_extremes(score, groups):
    require_lib()
    rng = np.random.default_rng(3)
    N, E, k = 96, 64, 6
    l = rng.standard_normal((N, E)).astype(np.float32)
    l[0] = -np.inf                                  # nothing left
    l[1] = -np.inf
    l[1, 63] = 0.5                                  # one expert left
    l[2] = np.nan
    l[3, ::2] = np.nan
    l[4:12][rng.random((8, E)) < 0.9] = -np.inf     # often fewer than k
    l[12:20] = np.round(l[12:20])                   # ties
    l[20] = 0.0
    l[21] = -0.0
    l[21, ::3] = 0.0
    l[22] = np.finfo(np.float32).min                # the lowest value is no mask
    l[23, 1:] = np.finfo(np.float32).min
    l[24] *= 40                                     # scores that underflow beside others
    l[25] = -100 + l[25]                            # sigmoids near the smallest numbers
    l[26] = -300 + l[26]
    l[27] = 90 + l[27]
    l[28] = 1e4 * l[28]
    up = rng.standard_normal((N, k)).astype(np.float32)
    for renorm in (True, False):
        check(l, None, up, k, score, *groups, 2, renorm, 1.5, ("masks", score, renorm))
    # with a bias only logits whose scores 64 bits tell apart
    l[24:29] = rng.standard_normal((5, E))
    for bias in (np.zeros(E), 0.3 * rng.standard_normal(E), np.full(E, -50.0)):
        check(l, bias.astype(np.float32), up, k, score, *groups, 2, True, 1.0, ("masks, bias", score))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups", [(1, 1), (4, 2)])
def test_near_ties_are_told_apart(score, groups):
    """Logits one step apart, the larger at the higher index: their scores, and
    the groups' strengths, are equal in 32 bits and not in 64."""
    require_lib()
    N, E, k = 40, 128, 9
    base = np.linspace(-2, 2, N).astype(np.float32)[:, None]
    steps = np.random.default_rng(0).permuted(np.tile(np.arange(E), (N, 1)), axis=1)
    l = (base.view(np.int32) + np.where(base < 0, -steps, steps).astype(np.int32)).view(np.float32)
    up = np.ones((N, k), np.float32)
    far = np.where(np.arange(E) % 2, 50.0, -49.0).astype(np.float32)  # sums of two, each with its own rounding
    for bias in (None, np.zeros(E, np.float32), np.full(E, 3.0, np.float32), far):
        check(l, bias, up, k, score, *groups, 2, True, 1.0, ("near", score, bias is None))
    # a few near pairs among ordinary rows, where the last slot and the next expert are the pair too
    r = np.random.default_rng(1)
    l = r.standard_normal((N, E)).astype(np.float32)
    bias = (0.1 * r.standard_normal(E)).astype(np.float32)
    for t in range(N):
        order = oracle.route_select(l[t:t + 1], E // 4, score, bias, *groups, 2)[0]
        i, j = order[t % 12], order[t % 12 + 1]
        bias_gap = np.float64(bias[j]) - np.float64(bias[i])
        if score == "sigmoid":  # j's score made i's less the biases' gap, up to rounding
            s = 1 / (1 + np.exp(-np.float64(l[t, i]))) - bias_gap
            if 0 < s < 1:
                l[t, j] = np.float32(np.log(s / (1 - s)))
        else:
            l[t, j] = l[t, i]
    for renorm in (True, False):
        check(l, bias, up, k, score, *groups, 2, renorm, 1.0, ("pairs", score))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups", [(64, (1, 1)), (64, (8, 2)), (512, (16, 3)), (256, (64, 2))])
def test_infinite_logits_still_give_distinct_experts(E, groups, score):
    require_lib()
    l = torch.randn(64, E, device=DEV)
    l[torch.rand(64, E, device=DEV) < 0.2] = float("inf")
    l[torch.rand(64, E, device=DEV) < 0.2] = float("-inf")
    l[torch.rand(64, E, device=DEV) < 0.1] = float("nan")
    for bias in (None, torch.randn(E, device=DEV)):
        for renorm in (True, False):
            plan = B.route_plan(64, E, 7, score, *groups, 2, renorm)
            idx, gates = B.route_forward(plan, l, bias)
            B.route_backward(plan, l, idx, torch.randn(64, 7, device=DEV))
            i = idx.cpu().numpy()
            assert i.min() >= 0 and i.max() < E and all(len(set(r)) == 7 for r in i.tolist())


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k,groups", [(64, 7, (1, 1)), (64, 7, (8, 2)), (512, 9, (16, 3)), (96, 40, (1, 1))])
def test_bias_that_is_not_finite_still_gives_distinct_experts(E, k, groups, score):
    require_lib()
    l = torch.randn(64, E, device=DEV)
    for bad in (float("nan"), float("inf"), float("-inf")):
        for share in (0.05, 0.5, 1.0):
            bias = torch.randn(E, device=DEV)
            bias[torch.rand(E, device=DEV) < share] = bad
            idx, _ = B.route_forward(B.route_plan(64, E, k, score, *groups, 2), l, bias)
            i = idx.cpu().numpy()
            assert i.min() >= 0 and i.max() < E and all(len(set(r)) == k for r in i.tolist()), (bad, share)


def test_unaligned_rows_other_stream_and_untouched_neighbours():
    require_lib()
    rng = np.random.default_rng(9)
    N, E, k = 21, 257, 5
    big = dev(rng.standard_normal((N + 2, E)).astype(np.float32))
    l = big[1:N + 1]  # contiguous, 4 bytes past a 16-byte step
    plan = B.route_plan(N, E, k, "sigmoid", renorm=False)
    ref = B.route_forward(plan, l.clone())
    up = dev(rng.standard_normal((N, k)).astype(np.float32))
    refd = B.route_backward(plan, l.clone(), ref[0], up)
    whole_i = torch.full((N + 2, k), -7, dtype=torch.int32, device=DEV)
    whole_g = torch.full((N + 2, k), -7.0, device=DEV)
    whole_d = torch.full((N + 2, E), -7.0, device=DEV)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    B.route_forward(plan, l, topk_idx=whole_i[1:N + 1], gates=whole_g[1:N + 1], stream=s)
    B.route_backward(plan, l, whole_i[1:N + 1], up, dlogits=whole_d[1:N + 1], stream=s)
    s.synchronize()
    assert torch.equal(whole_i[1:N + 1], ref[0]) and torch.equal(whole_g[1:N + 1], ref[1])
    assert torch.equal(whole_d[1:N + 1], refd)
    for w in (whole_i, whole_g, whole_d):
        assert bool((w[0] == -7).all()) and bool((w[-1] == -7).all())


def test_backward_ignores_entries_that_name_no_expert():
    require_lib()
    plan = B.route_plan(2, 8, 3, "sigmoid", renorm=True)
    l = torch.randn(2, 8, device=DEV)
    up = torch.randn(2, 3, device=DEV)
    idx = torch.tensor([[1, -1, 5], [900, 2, -2**31]], dtype=torch.int32, device=DEV)
    d = B.route_backward(plan, l, idx, up).cpu().numpy()
    sel = np.array([[1, 5], [2, 2]])
    ref = oracle.route_backward(l[:1].cpu().numpy(), sel[:1], up[:1, [0, 2]].cpu().numpy(), "sigmoid")
    assert np.allclose(d[0], ref[0], rtol=1e-5, atol=1e-7)
    assert np.allclose(d[1], 0, atol=1e-7)  # one expert renormalised to 1: no gradient


LAYER = {"tiny_f32": dict(N=256, c=64, flags=0), "train_bf16": dict(N=777, c=49, flags=0),
         "exact": dict(N=515, c=200, flags=1)}


@pytest.mark.parametrize("name", sorted(LAYER))
def test_layer_under_its_own_routing(name):
    """moe_routed_* under moe_bounded_forward's routing gives that layer's
    outputs bit for bit."""
    require_lib()
    cs = LAYER[name]
    wl = datagen.WORKLOADS["train_bf16" if name == "exact" else name]
    inp = datagen.Inputs(wl, N=cs["N"], dy=True)
    d = DevInputs(inp)
    plan = plan_for(wl, N=cs["N"], c=cs["c"])
    if cs["flags"]:
        B.moe_plan_set_flags(plan, cs["flags"])
    Y, idx, g, _, _ = B.moe_bounded_forward(plan, d.X, d.Wr, d.bias, d.Wg, d.Wu, d.Wd)
    ref = B.moe_bounded_backward(plan, d.X, d.Wr, d.Wg, d.Wu, d.Wd, d.dY, idx, g)
    Yr, st = B.moe_routed_forward(plan, d.X, d.Wg, d.Wu, d.Wd, idx, g)
    out = B.moe_routed_backward(plan, d.X, d.Wg, d.Wu, d.Wd, d.dY, idx, g)
    torch.cuda.synchronize()
    assert st["K"] == plan.K and st["dispatch_bytes"] <= st["dispatch_bound_bytes"]
    raw = lambda t: t.view(torch.int16) if t.dtype == torch.bfloat16 else t.view(torch.int32)
    assert torch.equal(raw(Y), raw(Yr))
    for n in ("dW_gate", "dW_up", "dW_down", "dgates"):
        assert torch.equal(raw(out[n]), raw(ref[n])), n
    # dX: the layer's, less its router's share
    share = ref["dlogits"].double() @ d.Wr.double().T
    want = dev_to_f64(ref["dX"]) - share.cpu().numpy()
    got = dev_to_f64(out["dX"])
    half = 2.0 ** -8 if d.X.dtype == torch.bfloat16 else 2.0 ** -22  # two roundings, and the sums' in fp32
    scale = np.abs(dev_to_f64(ref["dX"])) + np.abs(got) + 16 * np.abs(share.cpu().numpy())
    assert np.all(np.abs(got - want) <= half * scale + 1e-6 * np.abs(got).max())


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_graph_replays(score):
    require_lib()
    from test_gpu_graph import capture, replay_and_check
    plan = B.route_plan(301, 256, 8, score, 8, 4, 2, score == "sigmoid", 2.5)
    l, b, up = torch.randn(301, 256, device=DEV), torch.randn(256, device=DEV) * 0.1, torch.randn(301, 8, device=DEV)
    outs = {"idx": torch.empty((301, 8), dtype=torch.int32, device=DEV),
            "gates": torch.empty((301, 8), device=DEV), "dl": torch.empty((301, 256), device=DEV)}

    def call():
        B.route_forward(plan, l, b, outs["idx"], outs["gates"])
        B.route_backward(plan, l, outs["idx"], up, outs["dl"])

    call()
    torch.cuda.synchronize()
    refs = {k: t.clone() for k, t in outs.items()}
    replay_and_check("route " + score, capture(call), outs, refs)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k,groups", [(64, 8, (1, 1)), (64, 5, (8, 3)), (256, 8, (8, 4)), (512, 9, (16, 3)),
                                        (96, 20, (1, 1)), (24, 3, (1, 1))])
def test_nan_bias_masks_its_expert_among_near_ties(E, k, groups, score):
    """Few distinct logits and biases, so that equal and nearly equal scores are
    told apart in 64 bits; every group keeps experts enough.  A NaN bias then
    ranks as a bias far below all others, and its expert is never selected."""
    require_lib()
    rng = np.random.default_rng(E + k)
    l = (np.round(rng.standard_normal((200, E)) * 2) / 2).astype(np.float32)
    l = np.where(rng.random(l.shape) < 0.3, np.nextafter(l, np.float32(9)), l)
    bias = (0.125 * rng.integers(-1, 2, E)).astype(np.float32)
    for first, step in ((0, 2), (1, 2), (0, 4), (3, 8)):
        gone = np.zeros(E, bool)
        gone[first::step] = True
        per = E // groups[0]
        assert (~gone).reshape(-1, per).sum(1).min() >= 2 and (~gone).sum() * groups[1] // groups[0] >= k
        plan = B.route_plan(200, E, k, score, *groups, 2)
        idx, _ = B.route_forward(plan, dev(l), dev(np.where(gone, np.float32("nan"), bias)))
        want = oracle.route_select(l, k, score, np.where(gone, -1e30, bias), *groups, 2)
        got = idx.cpu().numpy()
        assert not gone[got].any(), (first, step)
        assert np.array_equal(got, want), (first, step)
