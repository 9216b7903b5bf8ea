"""The operators together, as a training step uses them: token embedding, layer
norm, routing by biased sigmoid scores in groups, the layer's experts under that
routing, a residual, layer norm, and distillation through the tied vocabulary
projection; then every gradient back to the leaves, the embedding's added onto
the projection's.

The reference is the same step in fp64 under torch's autograd, on the CPU, from
the same bf16 weights and with the step's own selection (its gates' gradient
does not flow through the choice).  Between a leaf and the loss a value is
rounded to bf16 at most 12 times (embedding, norm, expert rows, their SwiGLU
product, the layer's output, the residual, the second norm, and on the way back
the logit gradient, dX of the projection, of the norm, of the layer and of the
first norm), each by at most 2^-8 of itself, so 12 * 2^-8 bounds the relative
2-norm of what such roundings make of a gradient."""

import numpy as np
import pytest
import torch

import oracle
from gpu_common import DEV, B, needs_gpu, require_lib, say

pytestmark = [pytest.mark.gpu, needs_gpu]

N, V, H, F, E, K_EXP, K_LIST, T = 300, 1000, 256, 128, 16, 4, 8, 2.0
SCALE, GATE_SCALE, EPS = H ** 0.5, 2.5, 1e-5
TOL = 12 * 2.0 ** -8


class Step:
    def __init__(self, seed=0):
        g = torch.Generator().manual_seed(seed)
        bf = lambda *s, std: (std * torch.randn(*s, generator=g)).bfloat16().to(DEV)
        f32 = lambda *s, std, mean=0.0: (mean + std * torch.randn(*s, generator=g)).to(DEV)
        self.W = bf(V, H, std=0.05)
        self.Wr = f32(H, E, std=0.06)
        self.Wg, self.Wu, self.Wd = bf(E, H, F, std=0.06), bf(E, H, F, std=0.06), bf(E, F, H, std=0.08)
        self.g1, self.b1 = f32(H, std=0.1, mean=1.0), f32(H, std=0.1)
        self.g2, self.b2 = f32(H, std=0.1, mean=1.0), f32(H, std=0.1)
        self.balance = f32(E, std=0.05)
        ids = torch.randint(0, V, (N,), generator=g)
        ids[::7] = 3          # a common token
        ids[5::50] = -1       # padding
        self.ids = ids.int().to(DEV)
        self.t_idx = torch.randint(0, V, (N, K_LIST), generator=g).int().to(DEV)
        self.t_idx[11] = -1   # an ignored position
        self.t_logit = f32(N, K_LIST, std=2.0)
        self.dloss = torch.full((N,), 1.0 / N, device=DEV)
        self.pe = B.embed_plan(N, V, H, B.MOE_BF16, SCALE)
        self.pn = B.lnorm_plan(N, H, B.MOE_BF16, EPS)
        self.pr = B.route_plan(N, E, K_EXP, "sigmoid", 4, 2, 2, True, GATE_SCALE)
        self.pm = B.moe_plan_chunks(N, H, F, E, K_EXP, 64, 8, B.MOE_BF16)
        self.pk = B.kd_plan(N, H, V, 256, K_LIST, T)
        self.ws = {n: B.workspace(p, k, DEV) for n, p, k in (
            ("mf", self.pm, "fwd"), ("mb", self.pm, "bwd"), ("kd", self.pk, "both"), ("n1", self.pn, "bwd"),
            ("n2", self.pn, "bwd"), ("e", self.pe, "bwd"))}

    def run(self):
        ws = self.ws
        x0 = B.embed_forward(self.pe, self.W, self.ids)
        n1, m1, r1 = B.lnorm_forward(self.pn, x0, self.g1, self.b1)
        logits = n1.float() @ self.Wr
        idx, gates = B.route_forward(self.pr, logits, self.balance)
        y, _ = B.moe_routed_forward(self.pm, n1, self.Wg, self.Wu, self.Wd, idx, gates, ws=ws["mf"])
        x1 = x0 + y
        n2, m2, r2 = B.lnorm_forward(self.pn, x1, self.g2, self.b2)
        loss, lse, top = B.kd_forward(self.pk, n2, self.W, self.t_idx, self.t_logit, ws=ws["kd"])
        # back
        dn2, dW = B.kd_backward(self.pk, n2, self.W, self.t_idx, self.t_logit, lse, top, self.dloss, ws=ws["kd"])
        dx1, dg2, db2 = B.lnorm_backward(self.pn, x1, self.g2, dn2, m2, r2, ws=ws["n2"])
        moe = B.moe_routed_backward(self.pm, n1, self.Wg, self.Wu, self.Wd, dx1, idx, gates, ws=ws["mb"])
        dlogits = B.route_backward(self.pr, logits, idx, moe["dgates"])
        dn1 = (moe["dX"].float() + dlogits @ self.Wr.T).bfloat16()
        dWr = n1.float().T @ dlogits
        dx0, dg1, db1 = B.lnorm_backward(self.pn, x0, self.g1, dn1, m1, r1, ws=ws["n1"])
        dx0 = dx0 + dx1
        B.embed_backward(self.pe, self.ids, dx0, dW=dW, accumulate=True, ws=ws["e"])
        return dict(loss=loss, idx=idx, gates=gates, dW=dW, dWr=dWr, dW_gate=moe["dW_gate"], dW_up=moe["dW_up"],
                    dW_down=moe["dW_down"], dg1=dg1, db1=db1, dg2=dg2, db2=db2, logits=logits)

    def reference(self, idx):
        """Loss and gradients in fp64 with the selection idx."""
        d = lambda t: t.double().cpu().requires_grad_(True)
        W, Wr, Wg, Wu, Wd, g1, b1, g2, b2 = (d(t) for t in (self.W, self.Wr, self.Wg, self.Wu, self.Wd, self.g1, self.b1, self.g2, self.b2))
        ids = self.ids.cpu().long()
        x0 = torch.where((ids >= 0)[:, None], W[ids.clamp_min(0)] * SCALE, 0.0)

        def norm(x, g, b):
            c = x - x.mean(1, keepdim=True)
            return c / torch.sqrt((c * c).mean(1, keepdim=True) + EPS) * g + b

        n1 = norm(x0, g1, b1)
        s = torch.sigmoid(n1 @ Wr).gather(1, idx)
        gates = GATE_SCALE * s / s.sum(1, keepdim=True)
        y = torch.zeros_like(x0)
        for e in range(E):
            t, slot = (idx == e).nonzero(as_tuple=True)
            h = torch.nn.functional.silu(n1[t] @ Wg[e]) * (n1[t] @ Wu[e])
            y = y.index_add(0, t, (h @ Wd[e]) * gates[t, slot, None])
        n2 = norm(x0 + y, g2, b2)
        logq = torch.log_softmax(n2 @ W.T / T, 1)
        ti, tl = self.t_idx.cpu().long(), self.t_logit.double().cpu()
        p = torch.softmax(tl / T, 1)
        loss = T * T * torch.where(ti >= 0, p * (p.log() - logq.gather(1, ti.clamp_min(0))), 0.0).sum(1)
        (loss * self.dloss.double().cpu()).sum().backward()
        return dict(loss=loss.detach(), gates=gates.detach(), dW=W.grad, dWr=Wr.grad, dW_gate=Wg.grad, dW_up=Wu.grad,
                    dW_down=Wd.grad, dg1=g1.grad, db1=b1.grad, dg2=g2.grad, db2=b2.grad)


def test_step_against_autograd():
    require_lib()
    s = Step()
    out = s.run()
    torch.cuda.synchronize()
    idx = out["idx"].cpu().long()
    want = oracle.route_select(out["logits"].cpu().numpy(), K_EXP, "sigmoid", s.balance.cpu().numpy(), 4, 2, 2)
    assert np.array_equal(idx.numpy(), want)
    ref = s.reference(idx)
    off = {k: float((out[k].double().cpu() - r).norm() / r.norm()) for k, r in ref.items()}
    say("step: relative 2-norm errors", {k: f"{v:.1e}" for k, v in off.items()})
    assert all(v <= TOL for v in off.values()), off
    assert out["loss"][11] == 0


def test_step_repeats_on_another_stream_and_in_a_graph():
    """Bit for bit: eagerly twice, on a second stream, and as a captured graph
    replayed between eager steps; then on new inputs copied into its buffers."""
    require_lib()
    s = Step(1)
    keys = ("loss", "idx", "gates", "dW", "dWr", "dW_gate", "dW_up", "dW_down", "dg1", "db1", "dg2", "db2")
    ref = {k: v.clone() for k, v in s.run().items() if k in keys}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = s.run()
    side.synchronize()
    for k in keys:
        assert torch.equal(ref[k], other[k]), k
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = s.run()
    new = Step(2)
    for turn in range(4):
        if turn == 3:  # the graph reads its inputs when it runs
            for a in ("ids", "t_idx", "t_logit", "W"):
                getattr(s, a).copy_(getattr(new, a))
            ref = {k: v.clone() for k, v in s.run().items() if k in keys}
        for k in keys:
            out[k].fill_(7)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for k in keys:
            assert torch.equal(ref[k], out[k]), (turn, k)
        s.run()  # eager work on the same workspaces in between
        torch.cuda.synchronize()
