"""Pins of the fp64 distillation oracle: closed forms, torch's fp64 autograd
and finite differences."""

import numpy as np
import torch

import oracle


def case(N=7, H=6, V=20, K=5, seed=0):
    r = np.random.default_rng(seed)
    idx = np.stack([r.choice(V, K, replace=False) for _ in range(N)])
    return r.standard_normal((N, H)), r.standard_normal((V, H)), idx, 3 * r.standard_normal((N, K)), r.random(N)


def test_against_torch_with_short_empty_and_repeated_lists():
    X, W, idx, t, dl = case()
    idx[1, 3:] = -1
    idx[2] = 99
    t[3, 0] = -np.inf
    idx[4, 1] = idx[4, 0]
    for T in (1.0, 2.5):
        x, w = torch.tensor(X, requires_grad=True), torch.tensor(W, requires_grad=True)
        total = 0
        for n in range(len(X)):
            at = [j for j in range(5) if 0 <= idx[n, j] < 20 and t[n, j] > -np.inf]
            if not at:
                continue
            p = torch.softmax(torch.tensor(t[n, at]) / T, 0)
            logq = torch.log_softmax((x[n] @ w.T) / T, 0)
            loss = T * T * (p * (p.log() - logq[idx[n, at]])).sum()
            assert np.isclose(loss.item(), oracle.kd_forward(X, W, idx, t, T)[0][n], rtol=1e-12)
            total = total + dl[n] * loss
        total.backward()
        dX, dW = oracle.kd_backward(X, W, idx, t, T, dl)
        assert np.allclose(dX, x.grad.numpy(), rtol=1e-10, atol=1e-13)
        assert np.allclose(dW, w.grad.numpy(), rtol=1e-10, atol=1e-13)
        assert oracle.kd_forward(X, W, idx, t, T)[0][2] == 0 and not dX[2].any()


def test_matching_teacher_has_no_loss_and_no_gradient():
    X, W, _, _, dl = case(V=5)
    y = X @ W.T
    idx = np.tile(np.arange(5), (len(X), 1))
    loss, lse, y_top = oracle.kd_forward(X, W, idx, y + 3.0, 2.0)
    dX, dW = oracle.kd_backward(X, W, idx, y + 3.0, 2.0, dl)
    assert np.allclose(loss, 0, atol=1e-13) and np.allclose(y_top, y)
    assert np.allclose(dX, 0, atol=1e-13) and np.allclose(dW, 0, atol=1e-13)


def test_one_entry_is_cross_entropy():
    X, W, idx, t, dl = case(K=1)
    loss, lse, _ = oracle.kd_forward(X, W, idx, t, 1.0)
    ref, rlse = oracle.ce_forward(X, W, idx[:, 0].astype(np.int32))
    assert np.allclose(loss, ref) and np.allclose(lse, rlse)


def test_differences():
    X, W, idx, t, dl = case(N=2, H=3, V=9, K=4)
    dX, dW = oracle.kd_backward(X, W, idx, t, 1.7, dl)
    f = lambda x, w: oracle.kd_forward(x, w, idx, t, 1.7)[0] @ dl
    for a, d in ((X, dX), (W, dW)):
        for i in np.ndindex(a.shape):
            h = np.zeros_like(a)
            h[i] = 1e-6
            g = (f(X + h, W) - f(X - h, W)) if a is X else (f(X, W + h) - f(X, W - h))
            assert abs(g / 2e-6 - d[i]) < 1e-7
