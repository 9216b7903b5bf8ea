"""RMS norm with the residual's addition on the GPU against fp64 on the same inputs.

Tolerances, u = 2^-24 and e = half a step of the row type (bf16 2^-8, fp32 u).  A row sum of H <= 65536 terms runs at
most 256 deep in a lane and 9 across the work-group, so it is off by at most D u of the sum of its terms' sizes, D =
min(H, 256) + 12.
  S: one rounding of a sum of two numbers of the rows' type, so equal to the fp64 sum rounded once (bit for bit).
  rstd: the squares' sum, its roundings, the quotient by H and the root: relative (D + 8) u.
  Y: two products on that, then e once.  In 8 bits: half a step of e4m3 under the scale that the kernel chose, around
    the same; and the scale is the rule's for a largest magnitude within that error.
  dX: products of up to 4 roundings each on terms of their own size, the sum's and rstd's errors, then e once.
  dgamma: at most N / 512 + 1 terms in a lane, 512 / 4 + 4 in the fold."""

import numpy as np
import pytest
import torch

from gpu_common import DEV, B, dev_to_f64, needs_gpu, require_lib
from oracle import q8_oracle as Q

pytestmark = [pytest.mark.gpu, needs_gpu]
U = 2.0 ** -24
TYPES = {"bf16": (torch.bfloat16, 2.0 ** -8), "f32": (torch.float32, U)}


def inputs(N, H, dtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    dt = TYPES[dtype][0]
    x = torch.randn(N, H, generator=g) * (0.2 + torch.rand(H, generator=g) ** 4 * 6)
    r, dy, ds = (torch.randn(N, H, generator=g) for _ in range(3))
    return [t.to(dt).to(DEV) for t in (x, r, dy, ds)] + [(1 + 0.1 * torch.randn(H, generator=g)).to(DEV)]


def values8(q, s, H):
    """Values and scales [N][H] that the kernel's bytes stand for; the padding is looked at."""
    q, s = q.view(torch.uint8).cpu().numpy(), s.view(torch.uint8).cpu().numpy().astype(np.int64)
    blocks = -(-H // 128)
    assert np.all(s[:, blocks:] == 127) and np.all(q[:, H:] & 127 == 0)
    scale = np.repeat(2.0 ** (s[:, :blocks] - 127), 128, 1)[:, :H]
    return Q.decode(q[:, :H]) * scale, scale, s[:, :blocks] - 127


def check8(q, s, y, off):
    """8-bit rows against y known to |off|: each value within half a step of it, each scale the rule's."""
    got, scale, e = values8(q, s, y.shape[1])
    assert np.all(np.abs(got - y) <= Q.half_step(np.abs(y) + off, scale) + off), "values"
    top, slack = np.abs(Q.blocks(y)).max(2), Q.blocks(off).max(2)
    assert np.all((e >= Q.exponents(np.maximum(top - slack, 0))) & (e <= Q.exponents(top + slack))), "scales"


def check(N, H, dtype, residual, eps=1e-6, seed=0):
    x, r, dy, ds, gamma = inputs(N, H, dtype, seed)
    e = TYPES[dtype][1]
    plan = B.rms_plan(N, H, B.moe_dtype(x.dtype), eps)
    Y, S, rstd = B.rms_forward(plan, x, gamma, r if residual else None)
    Yq, Ys, S8, rstd8 = B.rms_forward_q8(plan, x, gamma, r if residual else None)
    dX, dgamma = B.rms_backward(plan, S, gamma, dy, rstd, ds if residual else None)
    torch.cuda.synchronize()
    assert torch.equal(S, (x.double() + r.double()).to(x.dtype) if residual else x)
    assert torch.equal(S8, S) and torch.equal(rstd8, rstd)
    if not residual:
        assert S is x and S8 is x
    s64, g64, dy64 = dev_to_f64(S), dev_to_f64(gamma), dev_to_f64(dy)
    y, rr = Q.rms(s64, g64, eps)
    D = (min(H, 256) + 12) * U
    r_rel = D + 8 * U
    assert np.all(np.abs(dev_to_f64(rstd) - rr) <= r_rel * rr), "rstd"
    off = (r_rel + 3 * U) * np.abs(y)
    assert np.all(np.abs(dev_to_f64(Y) - y) <= off * (1 + e) + e * np.abs(y)), "Y"
    check8(Yq, Ys, y, off)
    got = dev_to_f64(rstd)
    dx, dg = Q.rms_backward(s64, g64, dy64, got, dev_to_f64(ds) if residual else None)
    xh, d = np.abs(s64 * got[:, None]), np.abs(dy64 * g64)
    b = (xh * d).mean(1, keepdims=True)
    off = got[:, None] * (4 * U * d + xh * b * (D + 10 * U)) + 2 * U * np.abs(dx) + (2 * U * np.abs(dev_to_f64(ds)) if residual else 0)
    assert np.all(np.abs(dev_to_f64(dX) - dx) <= off * (1 + e) + e * np.abs(dx)), "dX"
    Dc = (N / 512 + 1 + 512 / 4 + 8) * U
    assert np.all(np.abs(dev_to_f64(dgamma) - dg) <= (Dc + 4 * U) * (np.abs(dy64) * xh).sum(0)), "dgamma"


SIZES = [(1, 1), (1, 2048), (3, 7), (777, 1111), (5, 64), (1, 65536), (9, 20000), (600, 512), (33, 7168), (5, 129), (257, 1024),
         (4, 16384), (3, 16392), (130, 2056), (2, 12000), (1025, 72), (7, 4096), (64, 5120), (3000, 256), (2, 65535)]


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("dtype", sorted(TYPES))
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "%dx%d" % s)
def test_against_oracle(size, dtype, residual):
    require_lib()
    check(*size, dtype, residual)


@pytest.mark.parametrize("dtype", sorted(TYPES))
def test_rows_of_zeros_and_of_extremes(dtype):
    """Rows of zeros (rstd is eps alone, a scale of 2^-110), tiny and large ones, one huge value among small ones."""
    x, _, dy, _, gamma = inputs(6, 300, dtype)
    x[0] = 0
    x[1] *= 1e-30
    x[2] *= 1e15
    x[3, 7] = 1e12
    x[4] = 0
    x[4, 299] = 1
    plan = B.rms_plan(6, 300, B.moe_dtype(x.dtype), 1e-6)
    q, s, _, rstd = B.rms_forward_q8(plan, x, gamma)
    dX, dgamma = B.rms_backward(plan, x, gamma, dy, rstd)
    torch.cuda.synchronize()
    y, r = Q.rms(dev_to_f64(x), dev_to_f64(gamma), 1e-6)
    check8(q, s, y, (256 + 24) * U * np.abs(y))
    assert bool((s.view(torch.uint8)[0, :3] == 17).all()) and bool(torch.isfinite(dX).all() and torch.isfinite(dgamma).all())


@pytest.mark.parametrize("H", [96, 1111, 7168, 20000])
def test_a_bad_row_spoils_itself_alone(H):
    x, r, dy, _, gamma = inputs(9, H, "bf16")
    plan = B.rms_plan(9, H)
    good = B.rms_forward_q8(plan, x, gamma, r)
    x[2, 5], x[6, H - 1] = float("nan"), float("inf")
    bad = B.rms_forward_q8(plan, x, gamma, r)
    torch.cuda.synchronize()
    keep = [0, 1, 3, 4, 5, 7, 8]
    for a, b in zip(good, bad):
        a, b = (t.view(torch.uint8) if t.dtype in (B.E4M3, B.E8M0) else t for t in (a, b))
        assert torch.equal(a[keep], b[keep])
    v = bad[0].float()
    assert torch.isnan(v[2, :H]).all() and torch.isnan(v[6, H - 1]) and torch.equal(v[:, H:], torch.zeros_like(v[:, H:]))


def test_outputs_over_inputs():
    """S over X or the residual, Y over X, dX over dY or dS: as with tensors of their own."""
    for H in (520, 1111, 20000):
        x, r, dy, ds, gamma = inputs(50, H, "bf16")
        plan = B.rms_plan(50, H)
        Y, S, rstd = B.rms_forward(plan, x, gamma, r)
        dX, dg = B.rms_backward(plan, S, gamma, dy, rstd, ds)
        for over_x in (True, False):
            a, b = x.clone(), r.clone()
            Y2, S2, r2 = B.rms_forward(plan, a, gamma, b, S=a if over_x else b, Y=None if over_x else a)
            assert torch.equal(Y, Y2) and torch.equal(S, S2) and torch.equal(rstd, r2)
            a, b = dy.clone(), ds.clone()
            dX2, dg2 = B.rms_backward(plan, S, gamma, a, rstd, b, dX=a if over_x else b)
            assert torch.equal(dX, dX2) and torch.equal(dg, dg2)
        a = x.clone()
        assert torch.equal(B.rms_forward(plan, a, gamma, Y=a)[0], B.rms_forward(plan, x, gamma)[0])


def test_rows_that_need_64_bit_offsets():
    """Rows past 2^31 elements: the last ones are as in a call of their own."""
    N, H = 70_000, 32_768
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB")
    x = torch.randn(64, H, device=DEV).bfloat16().repeat(N // 64 + 1, 1)[:N]
    gamma = torch.rand(H, device=DEV)
    last = slice(N - 32, N)
    q, s, _, rstd = B.rms_forward_q8(B.rms_plan(N, H), x, gamma)
    q2, s2, _, rstd2 = B.rms_forward_q8(B.rms_plan(32, H), x[last].contiguous(), gamma)
    assert torch.equal(q[last].view(torch.uint8), q2.view(torch.uint8)) and torch.equal(s[last].view(torch.uint8), s2.view(torch.uint8))
    assert torch.equal(rstd[last], rstd2)
    del q, s
    dX, _ = B.rms_backward(B.rms_plan(N, H), x, gamma, x, rstd)
    dX2, _ = B.rms_backward(B.rms_plan(32, H), x[last].contiguous(), gamma, x[last].contiguous(), rstd2)
    assert torch.equal(dX[last], dX2)


def test_no_rows():
    gamma = torch.ones(40, device=DEV)
    plan = B.rms_plan(0, 40)
    x = torch.empty(0, 40, dtype=torch.bfloat16, device=DEV)
    Y, S, rstd = B.rms_forward(plan, x, gamma)
    dX, dg = B.rms_backward(plan, x, gamma, x, rstd, dgamma=torch.full((40,), 7.0, device=DEV))
    assert Y.numel() == 0 and not dg.any()


@pytest.mark.parametrize("dtype", sorted(TYPES))
def test_values_next_to_borders(dtype):
    """Values next to where e4m3 or a scale turn are formed in 64 bits from the row's sum, whose fp32 part (eight products a
    chain, up to four such, four steps over 16 lanes) is off by 16 u at most, u = 2^-24: rstd by 8 u.  Of values spread over
    their logarithm, 8 borders an octave have 8 * 2 * 8 u / ln 2 = 185 u within that: 46 of 2048 x 2048.  (fp32 products
    would be off by another 2 u to 5 u; a value on the wrong side is one step away, never more.)"""
    require_lib()
    N = H = 2048
    g = torch.Generator().manual_seed(9)
    x = torch.randn(N, H, generator=g).to(TYPES[dtype][0]).to(DEV)
    gamma = (1 + 0.1 * torch.randn(H, generator=g)).to(DEV)
    plan = B.rms_plan(N, H, B.moe_dtype(x.dtype), 1e-6)
    q, s, _, _ = B.rms_forward_q8(plan, x, gamma)
    v = dev_to_f64(x)
    y = v / np.sqrt(np.mean(v * v, axis=1, keepdims=True) + float(np.float32(1e-6))) * dev_to_f64(gamma)
    want, e = Q.quantise(y)
    got, _, ge = values8(q, s, H)
    assert np.array_equal(ge, e)
    assert int((got != want).sum()) <= 46
    assert (np.abs(got - want) <= np.exp2(np.floor(np.log2(np.maximum(np.abs(want), 1e-30))) - 3)).all()


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("dtype", sorted(TYPES))
def test_wide_rows_next_to_borders(dtype, residual):
    """Rows past 16,384 columns are summed in 64 bits throughout, so that values formed in 64 bits are those of the fp64
    norm: all numbers and scales.  (From sums in 32 bits up to three of four million are not.)"""
    require_lib()
    N, H = 200, 20_000
    g = torch.Generator().manual_seed(10)
    x, r = (torch.randn(N, H, generator=g).to(TYPES[dtype][0]).to(DEV) for _ in range(2))
    gamma = (1 + 0.1 * torch.randn(H, generator=g)).to(DEV)
    q, s, S, _ = B.rms_forward_q8(B.rms_plan(N, H, B.moe_dtype(x.dtype), 1e-6), x, gamma, r if residual else None)
    v = dev_to_f64(S)
    y = v / np.sqrt(np.mean(v * v, axis=1, keepdims=True) + float(np.float32(1e-6))) * dev_to_f64(gamma)
    want, e = Q.quantise(y)
    got, _, ge = values8(q, s, H)
    assert np.array_equal(ge, e) and int((got != want).sum()) == 0
