"""Pins of the fp64 routing oracle: closed forms, torch's fp64 autograd and
finite differences."""

import numpy as np
import pytest
import torch

import oracle


def draw(N, E, seed=0):
    return np.random.default_rng(seed).standard_normal((N, E))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_gates_and_gradient_against_torch(score, renorm):
    l = draw(9, 12)
    idx = oracle.route_select(l, 4, score, np.linspace(-0.2, 0.2, 12))
    t = torch.tensor(l, requires_grad=True)
    s = torch.softmax(t, 1) if score == "softmax" else torch.sigmoid(t)
    sel = s.gather(1, torch.tensor(idx))
    g = 2.5 * (sel / sel.sum(1, keepdim=True) if renorm else sel)
    up = draw(9, 4, 1)
    (g * torch.tensor(up)).sum().backward()
    assert np.allclose(oracle.route_gates(l, idx, score, renorm, 2.5), g.detach().numpy(), rtol=1e-13, atol=0)
    assert np.allclose(oracle.route_backward(l, idx, up, score, renorm, 2.5), t.grad.numpy(), rtol=1e-11, atol=1e-14)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_gradient_against_differences(score, renorm):
    l, up = draw(3, 8), draw(3, 3, 2)
    idx = oracle.route_select(l, 3, score)
    f = lambda x: (oracle.route_gates(x, idx, score, renorm, 1.5) * up).sum()
    d = oracle.route_backward(l, idx, up, score, renorm, 1.5)
    for t in range(3):
        for e in range(8):
            h = np.zeros_like(l)
            h[t, e] = 1e-5
            assert abs((f(l + h) - f(l - h)) / 2e-5 - d[t, e]) < 1e-8


def test_selection_brute_force_and_ties():
    l = np.round(draw(50, 16) * 2) / 2  # many ties
    idx = oracle.route_select(l, 5, "sigmoid")
    assert np.array_equal(idx, np.argsort(-l, axis=1, kind="stable")[:, :5])
    # bias moves the selection, not the gates
    b = np.zeros(16)
    b[3] = 10.0
    idb = oracle.route_select(l, 5, "sigmoid", b)
    assert np.all(idb[:, 0] == 3)
    g = oracle.route_gates(l, idb, "sigmoid", False, 1.0)
    assert np.allclose(g[:, 0], 1 / (1 + np.exp(-l[:, 3])))


def test_groups_keep_the_strongest():
    l = np.full((1, 8), -1.0)
    l[0, 0] = 3.0                 # group 0: one strong expert
    l[0, 2:4] = 1.5               # group 1: two good ones
    two = oracle.route_select(l, 2, "sigmoid", n_group=4, topk_group=1, group_top=2)
    one = oracle.route_select(l, 2, "sigmoid", n_group=4, topk_group=1, group_top=1)
    assert list(two[0]) == [2, 3] and list(one[0]) == [0, 1]


def test_masked_rows():
    l = np.full((2, 6), -np.inf)
    l[1, 4] = 0.0
    l[1, 5] = np.nan
    for score in ("softmax", "sigmoid"):
        idx = oracle.route_select(l, 3, score)
        assert list(idx[0]) == [0, 1, 2] and list(idx[1]) == [4, 0, 1]
        for renorm in (True, False):
            g = oracle.route_gates(l, idx, score, renorm)
            assert np.all(g[0] == 0) and np.all(g[1, 1:] == 0) and g[1, 0] > 0
            assert np.all(oracle.route_backward(l, idx, np.ones((2, 3)), score, renorm)[0] == 0)
