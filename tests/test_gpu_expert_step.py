"""The 8-bit path of an expert layer as a training step uses it: RMS norm of the residual's sum into 8-bit rows, routing
by scores, the rows of each expert gathered, gate and up products in 8 bits, SwiGLU with its checkpoint in 8 bits, the
down product, the weighted sum onto the residual; then every gradient back, the weight gradients from the rows kept in
8 bits, the data gradients through products in 8 bits.  And the same step in bfloat16.

The reference is the step in fp64 under torch's autograd, on the CPU, from the same weights and under the step's own
routing.  Between a leaf and a gradient a value is rounded to e4m3 at most 8 times (the norm's output, three matrices,
a or u, h, and on the way back dy and one of da, du), each by at most 2^-4 of itself or half the block's smallest
number (2^-10 of a scale that is at most 2^-8 of the block's largest: 2^-17 of it, nothing beside the rest), so
8 * 2^-4 bounds the relative 2-norm of what such roundings make of a gradient to first order; in bfloat16 at most 12
roundings of 2^-8."""

import numpy as np
import pytest
import torch

from gpu_common import DEV, B, dev_to_f64, needs_gpu, require_lib, say
from oracle import q8_oracle as Q
from test_gpu_gmm import TRUNC, close
from test_gpu_rms import check8, values8

pytestmark = [pytest.mark.gpu, needs_gpu]

N, H, F, E, K = 300, 264, 136, 16, 4
EPS = 1e-6
LEAVES = ("x", "gamma", "Wg", "Wu", "Wd")


class Step:
    def __init__(self, seed=0, eight=True):
        g = torch.Generator().manual_seed(seed)
        bf = lambda *s, std: (std * torch.randn(*s, generator=g)).bfloat16().to(DEV)
        self.eight = eight
        self.x, self.r, self.dout = bf(N, H, std=1.0), bf(N, H, std=0.5), bf(N, H, std=1.0)
        self.gamma = (1 + 0.1 * torch.randn(H, generator=g)).to(DEV)
        self.Wg, self.Wu, self.Wd = bf(E, H, F, std=0.06), bf(E, H, F, std=0.06), bf(E, F, H, std=0.08)
        logits = torch.randn(N, E, generator=g).to(DEV)
        self.idx, self.gates = B.route_forward(B.route_plan(N, E, K, "sigmoid"), logits)
        # the pairs by expert, as a program's own dispatch has them
        self.order = self.idx.flatten().long().argsort(stable=True)
        self.token, self.back = self.order // K, self.order.argsort()
        self.offsets = torch.nn.functional.pad(torch.bincount(self.idx.flatten().long(), minlength=E).cumsum(0), (1, 0)).int()
        R, ops = N * K, B.GMM_Q8 if eight else B.GMM_BF16
        self.norm = B.rms_plan(N, H, B.MOE_BF16, EPS)
        self.up, self.down = B.gmm_plan(R, H, F, E, ops), B.gmm_plan(R, F, H, E, ops)
        self.rows_h, self.rows_f = B.q8_plan(R, H), B.q8_plan(R, F)
        if eight:  # along K for the forward products, along N for dX
            self.wg, self.wu, self.wd = (B.q8_pack_weights(w) for w in (self.Wg, self.Wu, self.Wd))
        self.ws = {p: B.workspace(getattr(self, p), "both" if p != "norm" else "bwd", DEV) for p in ("up", "down", "norm")}

    def take(self, t):
        if t.dtype in (B.E4M3, B.E8M0):
            return t.view(torch.uint8)[self.token].view(t.dtype)
        return t[self.token]

    def run(self):
        off, ws, up, down = self.offsets, self.ws, self.up, self.down
        g = self.gates.flatten()[self.order][:, None]
        if self.eight:
            nq, ns, S, rstd = B.rms_forward_q8(self.norm, self.x, self.gamma, self.r)
            xq, xs = self.take(nq), self.take(ns)
            a = B.gmm8_forward(up, xq, xs, *self.wg[:2], off, ws=ws["up"])
            u = B.gmm8_forward(up, xq, xs, *self.wu[:2], off, ws=ws["up"])
            hq, hs, kept = B.q8_swiglu_forward(self.rows_f, a, u)
            y = B.gmm8_forward(down, hq, hs, *self.wd[:2], off, ws=ws["down"])
        else:
            n, S, rstd = B.rms_forward(self.norm, self.x, self.gamma, self.r)
            xr = self.take(n)
            a, u = B.gmm_forward(up, xr, self.Wg, off, ws=ws["up"]), B.gmm_forward(up, xr, self.Wu, off, ws=ws["up"])
            h = (torch.nn.functional.silu(a.float()) * u.float()).bfloat16()
            y = B.gmm_forward(down, h, self.Wd, off, ws=ws["down"])
        out = (S.float() + (y.float() * g)[self.back].view(N, K, H).sum(1)).bfloat16()
        # back
        dy = (self.take(self.dout).float() * g).bfloat16()
        if self.eight:
            dh = B.gmm8_forward(up, *B.q8_pack(self.rows_h, dy), *self.wd[2:], off, ws=ws["up"])
            dWd = B.gmm8_backward_dw(down, hq, hs, dy, off, ws=ws["down"])
            da, du = B.q8_swiglu_backward(self.rows_f, kept, dh)
            dWg, dWu = (B.gmm8_backward_dw(up, xq, xs, d, off, ws=ws["up"]) for d in (da, du))
            dx1 = B.gmm8_forward(down, *B.q8_pack(self.rows_f, da), *self.wg[2:], off, ws=ws["down"])
            dx2 = B.gmm8_forward(down, *B.q8_pack(self.rows_f, du), *self.wu[2:], off, ws=ws["down"])
        else:
            dh = B.gmm_backward_dx(down, dy, self.Wd, off, ws=ws["down"])
            dWd = B.gmm_backward_dw(down, h, dy, off, ws=ws["down"])
            af, uf, d = a.float(), u.float(), dh.float()
            sg = torch.sigmoid(af)
            da, du = (d * uf * sg * (1 + af * (1 - sg))).bfloat16(), (d * af * sg).bfloat16()
            dWg, dWu = (B.gmm_backward_dw(up, xr, t, off, ws=ws["up"]) for t in (da, du))
            dx1, dx2 = B.gmm_backward_dx(up, da, self.Wg, off, ws=ws["up"]), B.gmm_backward_dx(up, du, self.Wu, off, ws=ws["up"])
        dn = (dx1.float() + dx2.float())[self.back].view(N, K, H).sum(1).bfloat16()
        dx, dgamma = B.rms_backward(self.norm, S, self.gamma, dn, rstd, self.dout, ws=ws["norm"])
        return dict(out=out, x=dx, gamma=dgamma, Wg=dWg, Wu=dWu, Wd=dWd)

    def reference(self):
        d = {n: getattr(self, n).double().cpu().requires_grad_(True) for n in LEAVES}
        S = d["x"] + self.r.double().cpu()
        n = S / torch.sqrt((S * S).mean(1, keepdim=True) + EPS) * d["gamma"]
        idx, gates = self.idx.cpu().long(), self.gates.double().cpu()
        y = torch.zeros_like(S)
        for e in range(E):
            t, slot = (idx == e).nonzero(as_tuple=True)
            h = torch.nn.functional.silu(n[t] @ d["Wg"][e]) * (n[t] @ d["Wu"][e])
            y = y.index_add(0, t, (h @ d["Wd"][e]) * gates[t, slot, None])
        out = S + y
        (out * self.dout.double().cpu()).sum().backward()
        return dict({k: v.grad for k, v in d.items()}, out=out.detach())


@pytest.mark.parametrize("eight", [True, False], ids=["8 bits", "bf16"])
def test_step_against_autograd(eight):
    require_lib()
    s = Step(eight=eight)
    out, ref = s.run(), s.reference()
    torch.cuda.synchronize()
    off = {k: float((out[k].double().cpu() - r).norm() / r.norm()) for k, r in ref.items()}
    say("expert step: relative 2-norm errors", {k: f"{v:.1e}" for k, v in off.items()})
    tol = 8 * 2.0 ** -4 if eight else 12 * 2.0 ** -8
    assert all(v <= tol for v in off.values()), off


@pytest.mark.parametrize("eight", [True, False], ids=["8 bits", "bf16"])
def test_step_repeats_on_another_stream_and_in_a_graph(eight):
    """Bit for bit: eagerly twice, on a second stream, and as a captured graph replayed between eager steps; then on new
    inputs copied into its buffers."""
    require_lib()
    s = Step(1, eight)
    ref = {k: v.clone() for k, v in s.run().items()}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = s.run()
    side.synchronize()
    for k in ref:
        assert torch.equal(ref[k], other[k]), k
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = s.run()
    new = Step(2, eight)
    for turn in range(4):
        if turn == 3:  # the graph reads its inputs when it runs
            for a in ("x", "r", "dout", "gamma"):
                getattr(s, a).copy_(getattr(new, a))
            ref = {k: v.clone() for k, v in s.run().items()}
        for v in out.values():
            v.fill_(7)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for k in ref:
            assert torch.equal(ref[k], out[k]), (turn, k)
        s.run()  # eager work on the same workspaces in between
        torch.cuda.synchronize()


def test_a_step_on_another_stream_by_argument():
    """Calls given a stream run and allocate there, whatever stream is current."""
    s = Step(3)
    want = B.rms_forward_q8(s.norm, s.x, s.gamma, s.r)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = B.rms_forward_q8(s.norm, s.x, s.gamma, s.r, stream=side)
    xq, xs = s.take(want[0]), s.take(want[1])
    torch.cuda.synchronize()
    a = B.gmm8_forward(s.up, xq, xs, *s.wg[:2], s.offsets, stream=side)
    kept = B.q8_swiglu_forward(s.rows_f, a, a, stream=side)[2]
    da, _ = B.q8_swiglu_backward(s.rows_f, kept, a, stream=side)
    dw = B.gmm8_backward_dw(s.up, xq, xs, da, s.offsets, stream=side)
    side.synchronize()
    for x, y in zip(want, got):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    a2 = B.gmm8_forward(s.up, xq, xs, *s.wg[:2], s.offsets)
    da2, _ = B.q8_swiglu_backward(s.rows_f, B.q8_swiglu_forward(s.rows_f, a2, a2)[2], a2)
    assert torch.equal(a, a2) and torch.equal(da, da2) and torch.equal(dw, B.gmm8_backward_dw(s.up, xq, xs, da2, s.offsets))


U, E16 = 2.0 ** -24, 2.0 ** -8


@pytest.mark.parametrize("eight", [True, False], ids=["8 bits", "bf16"])
def test_step_beside_the_residual(eight):
    """As test_step_against_autograd, of what the experts add to out and to dx, which the residual's S and dout hide there,
    and with the roundings of a value taken as independent: of numbers spread over their logarithm one to e4m3 is off by
    2^-4 sqrt(0.54 / 3) (uniform in its cell, 0.54 the mean of 1 / m^2), eight by 0.075, twelve to bfloat16 by 0.0057; the
    bound is twice that, and the two roundings of the whole out, or of the whole dx.  (In fp64 a step whose dA has no
    1 + a (1 - g) is 0.18 to 0.25 off in dx, dgamma and dWg, one without its up product's share of dx 0.69 to 0.73.)"""
    require_lib()
    s = Step(eight=eight)
    out, ref = s.run(), s.reference()
    torch.cuda.synchronize()
    x, r, dout = (getattr(s, n).double().cpu() for n in ("x", "r", "dout"))
    tol = 2 * (8 ** 0.5 * 2.0 ** -4 if eight else 12 ** 0.5 * E16) * (0.54 / 3) ** 0.5
    off = {}
    for k, v in ref.items():
        rest = {"out": x + r, "x": dout}.get(k, torch.zeros(()))
        part = (v - rest).norm()
        off[k] = float((out[k].double().cpu() - v).norm() / part), tol + (2 * E16 * float(v.norm() / part) if k in ("out", "x") else 0.0)
    say("expert step beside the residual: relative 2-norm errors", {k: "%.1e of %.1e" % v for k, v in off.items()})
    assert all(v <= t for v, t in off.values()), off


class Calls:
    """Every call that the step makes, with its arguments and what it returned."""

    NAMES = ("rms_forward", "rms_forward_q8", "rms_backward", "q8_pack", "q8_swiglu_forward", "q8_swiglu_backward", "gmm_forward",
             "gmm_backward_dx", "gmm_backward_dw", "gmm8_forward", "gmm8_backward_dw")

    def __init__(self, monkeypatch):
        self.made = []
        for name in self.NAMES:
            monkeypatch.setattr(B, name, self.recorded(name, getattr(B, name)))

    def recorded(self, name, f):
        def call(plan, *args, **kw):
            out = f(plan, *args, **kw)
            self.made.append((name, plan, args, out))
            return out
        return call


def weights64(q, s, cols):
    """Values [E][rows][cols] of weights in 8 bits."""
    e = torch.exp2(s.view(torch.uint8)[:, :, :-(-cols // 128)].double() - 127)
    return q[:, :, :cols].double() * e.repeat_interleave(128, 1)[:, :q.shape[1]].repeat_interleave(128, 2)[:, :, :cols]


def rows64(q, s, cols):
    return torch.from_numpy(values8(q, s, cols)[0]).to(DEV)


def by_row(x, w, offsets):
    """Rows of each expert by its matrix [E][columns summed][columns], and by magnitudes."""
    o = offsets.tolist()
    parts = [(x[o[e]:o[e + 1]], w[e].contiguous()) for e in range(len(o) - 1)]
    return torch.cat([a @ b for a, b in parts]), torch.cat([a.abs() @ b.abs() for a, b in parts])


def by_matrix(x, d, offsets):
    o = offsets.tolist()
    parts = [(x[o[e]:o[e + 1]].T.contiguous(), d[o[e]:o[e + 1]]) for e in range(len(o) - 1)]
    return torch.stack([a @ b for a, b in parts]), torch.stack([a.abs() @ b.abs() for a, b in parts])


def check_call(name, plan, a, out):
    if name in ("gmm_forward", "gmm_backward_dx"):
        ref, size = by_row(a[0].double(), a[1].double() if name == "gmm_forward" else a[1].double().transpose(1, 2), a[2])
        close(out, ref, size, max(plan.K, plan.N), E16, name)
    elif name == "gmm8_forward":
        ref, size = by_row(rows64(a[0], a[1], plan.K), weights64(a[2], a[3], plan.K).transpose(1, 2), a[4])
        close(out, ref, size, plan.K, E16, name, TRUNC)
    elif name in ("gmm_backward_dw", "gmm8_backward_dw"):
        x, d, off = (a[0].double(), a[1], a[2]) if name == "gmm_backward_dw" else (rows64(a[0], a[1], plan.K), a[2], a[3])
        ref, size = by_matrix(x, d.double(), off)
        close(out, ref, size, plan.R, 0, name)
    elif name in ("rms_forward", "rms_forward_q8"):
        S, rstd = out[-2:]
        assert torch.equal(S, (a[0].double() + a[2].double()).bfloat16())
        y, r = Q.rms(dev_to_f64(S), dev_to_f64(a[1]), EPS)
        off = (256 + 24) * U
        assert np.all(np.abs(dev_to_f64(rstd) - r) <= off * r)
        if name == "rms_forward":
            assert np.all(np.abs(dev_to_f64(out[0]) - y) <= (off + E16) * np.abs(y))
        else:
            check8(out[0], out[1], y, off * np.abs(y))
    elif name == "rms_backward":
        S, gamma, dy, r, ds = (dev_to_f64(t) for t in a[:5])
        dx, dg = Q.rms_backward(S, gamma, dy, r, ds)
        xh, d = np.abs(S * r[:, None]), np.abs(dy * gamma)
        inner = r[:, None] * (d + xh * (xh * d).mean(1, keepdims=True))
        assert np.all(np.abs(dev_to_f64(out[0]) - dx) <= E16 * np.abs(dx) + (256 + 24) * U * (inner + np.abs(ds)))
        assert np.all(np.abs(dev_to_f64(out[1]) - dg) <= (256 + 24) * U * (np.abs(dy) * xh).sum(0))
    elif name == "q8_pack":
        assert np.array_equal(values8(*out, plan.H)[0], Q.quantise(dev_to_f64(a[0]))[0])
    elif name == "q8_swiglu_forward":
        g, u = dev_to_f64(a[0]), dev_to_f64(a[1])
        assert np.array_equal(values8(*out[:2], plan.H)[0], Q.quantise(Q.swiglu(g, u))[0])
        for pair, x in ((out[2][:2], g), (out[2][2:], u)):
            assert np.array_equal(values8(*pair, plan.H)[0], Q.quantise(x)[0])
    elif name == "q8_swiglu_backward":
        g, u, d = values8(*a[0][:2], plan.H)[0], values8(*a[0][2:], plan.H)[0], dev_to_f64(a[1])
        t, terms = np.abs(g), np.abs(d * u) / (1 + np.exp(-g))
        for x, ref, size in zip(out, Q.swiglu_backward(g, u, d), (terms * (1 + t), 0.0)):
            assert np.all(np.abs(dev_to_f64(x) - ref) <= E16 * np.abs(ref) + (16 + 2 * t) * U * (np.abs(ref) + size))
    else:
        raise AssertionError(name)


@pytest.mark.parametrize("eight", [True, False], ids=["8 bits", "bf16"])
def test_every_call_of_the_step(eight, monkeypatch):
    """Each call's outputs against the formula in fp64 on the values that this call was given, to the bounds of the
    operators' own tests: a term that is left out anywhere is far outside (the mean of the norm's gradient is 0.1 of dx)."""
    require_lib()
    s = Step(4, eight)
    calls = Calls(monkeypatch)
    out = s.run()
    torch.cuda.synchronize()
    for c in calls.made:
        check_call(*c)
    names = [c[0] for c in calls.made]
    assert len(names) == (16 if eight else 11)
    # the sum onto the residual: fp32 sums of K terms, rounded once
    first, y = calls.made[0], [c[3] for c in calls.made if c[0] in ("gmm8_forward", "gmm_forward")][2]
    S, g = first[3][-2].double(), s.gates.flatten()[s.order][:, None].double()
    terms = (y.double() * g)[s.back].view(N, K, H)
    want, size = S + terms.sum(1), S.abs() + terms.abs().sum(1)
    assert bool(((out["out"].double() - want).abs() <= E16 * want.abs() + 8 * U * size).all())
