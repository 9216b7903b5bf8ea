"""Pins of the oracle of rows in 8 bits, and of the gradients that go with them, on the CPU."""

import numpy as np
import pytest
import torch

import oracle
from oracle import q8_oracle as Q


def test_table_is_e4m3():
    codes = torch.arange(256, dtype=torch.uint8)
    assert np.array_equal(Q.decode(codes.numpy()), codes.view(torch.float8_e4m3fn).double().numpy(), equal_nan=True)
    assert Q.TABLE[-1] == 448 and Q.TABLE[1] == 2.0 ** -9


def test_nearest_is_the_cast():
    """Every fp32 value with three mantissa bits to spare around each number, both signs, and random ones."""
    t = Q.TABLE
    mid = (t[1:] + t[:-1]) / 2
    x = np.concatenate([t, mid, mid * (1 - 2.0 ** -20), mid * (1 + 2.0 ** -20), np.random.default_rng(0).uniform(0, 448, 5000)])
    x = np.concatenate([x, -x]).astype(np.float32)
    assert np.array_equal(Q.nearest(x.astype(np.float64)), torch.from_numpy(x).to(torch.float8_e4m3fn).double().numpy())


def test_scale_is_the_smallest():
    for a in (448.0, np.nextafter(448.0, 500), 447.9, 1.0, 1.75, np.nextafter(1.75, 2), 2.0 ** -100, 3e38, 2.0 ** 127):
        e = int(Q.exponents(a))
        assert a / 2.0 ** e <= 448 < a / 2.0 ** (e - 1), a
    assert Q.exponents(0.0) == -110 and Q.exponents(2.0 ** -140) == -110


def test_rounding_is_at_most_half_a_step():
    x = np.random.default_rng(1).normal(size=(40, 300)) * np.exp(np.random.default_rng(2).normal(size=(40, 1)) * 5)
    q, e = Q.quantise(x)
    s = np.repeat(2.0 ** e, 128, 1)[:, :300]
    assert np.all(np.abs(q - x) <= Q.half_step(x, s))
    assert np.all(np.abs(q - x) <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * s))


@pytest.mark.parametrize("which", ["swiglu", "rms", "rms with the residual's gradient"])
def test_gradients_against_differences_and_autograd(which):
    g = np.random.default_rng(3)
    a, u, d = (g.normal(size=(5, 7)) for _ in range(3))
    t = lambda x: torch.from_numpy(x).requires_grad_(True)
    h = 1e-6
    if which == "swiglu":
        f = lambda a, u: (Q.swiglu(a, u) * d).sum()
        got = Q.swiglu_backward(a, u, d)
        ta, tu = t(a), t(u)
        (torch.nn.functional.silu(ta) * tu * torch.from_numpy(d)).sum().backward()
        leaves, auto = [a, u], [ta.grad, tu.grad]
    else:
        gamma, ds = g.normal(size=7), (g.normal(size=(5, 7)) if "residual" in which else None)
        f = lambda x, w: (Q.rms(x, w, 1e-3)[0] * d).sum() + (0 if ds is None else (x * ds).sum())
        got = Q.rms_backward(a, gamma, d, Q.rms(a, gamma, 1e-3)[1], ds)
        ta, tg = t(a), t(gamma)
        loss = (torch.nn.functional.rms_norm(ta, (7,), tg, 1e-3) * torch.from_numpy(d)).sum()
        if ds is not None:
            loss = loss + (ta * torch.from_numpy(ds)).sum()
        loss.backward()
        leaves, auto = [a, gamma], [ta.grad, tg.grad]
    for i, (x, gx, ax) in enumerate(zip(leaves, got, auto)):
        assert np.allclose(gx, ax.numpy(), rtol=1e-10, atol=1e-12)
        for at in np.ndindex(x.shape):
            lo, hi = [y.copy() for y in leaves], [y.copy() for y in leaves]
            lo[i][at] -= h
            hi[i][at] += h
            assert abs((f(*hi) - f(*lo)) / (2 * h) - gx[at]) <= 1e-7 * (1 + abs(gx[at]))


def test_weights_share_a_scale_per_block():
    w = np.random.default_rng(4).normal(size=(2, 130, 140))
    q, e = Q.quantise_weights(w)
    assert e.shape == (2, 2, 2)
    for i in range(2):
        for kb in range(2):
            for nb in range(2):
                part = w[i, kb * 128:(kb + 1) * 128, nb * 128:(nb + 1) * 128]
                assert e[i, kb, nb] == Q.exponents(np.abs(part).max())
                assert np.array_equal(q[i, kb * 128:(kb + 1) * 128, nb * 128:(nb + 1) * 128], Q.nearest(part / 2.0 ** e[i, kb, nb]) * 2.0 ** e[i, kb, nb])
    assert oracle.q8_oracle is Q
