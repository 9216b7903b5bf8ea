"""Rows in 8 bits and SwiGLU with 8-bit checkpoints on the GPU against fp64 on the same inputs.

Packing rounds once from the given values, so numbers and scales equal the oracle's; unpacking to bfloat16 is exact.
SwiGLU, u = 2^-24: 1 / (1 + e^-a) through a hardware exponential of a log2(e), whose rounded argument alone moves it by
|a| u; that, the exponential, sum, quotient and products leave h off by at most (8 + |a|) u of itself (and 2^-120 where
the exponential passes the type's range), so does dU; dA has the factor 1 + a (1 - g), off by |a| (6 + |a|) u and 4 u of
its terms.  Then half a step of the output's type: e4m3 under the kernel's scale, or bf16 2^-8, fp32 u."""

import numpy as np
import pytest
import torch

from gpu_common import DEV, B, dev_to_f64, needs_gpu, require_lib
from oracle import q8_oracle as Q
from test_gpu_rms import TYPES, check8, values8

pytestmark = [pytest.mark.gpu, needs_gpu]
U = 2.0 ** -24
SIZES = [(1, 1), (1, 128), (3, 7), (5, 129), (777, 1111), (2, 65536), (64, 512), (33, 640), (1000, 72), (1, 4096), (4097, 136), (0, 5)]


def rows(N, H, dtype, seed=0, spread=3.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(N, H, generator=g) * torch.exp(spread * torch.randn(N, 1, generator=g))).to(TYPES[dtype][0]).to(DEV)


@pytest.mark.parametrize("dtype", sorted(TYPES))
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "%dx%d" % s)
def test_pack_and_unpack(size, dtype):
    require_lib()
    N, H = size
    x = rows(N, H, dtype)
    plan = B.q8_plan(N, H, B.moe_dtype(x.dtype))
    q, s = B.q8_pack(plan, x)
    back = B.q8_unpack(plan, q, s)
    torch.cuda.synchronize()
    if N == 0:
        return
    want, e = Q.quantise(dev_to_f64(x))
    got, _, ge = values8(q, s, H)
    assert np.array_equal(ge, e) and np.array_equal(got, want)
    assert np.array_equal(dev_to_f64(back), want)
    assert np.array_equal(dev_to_f64(B.q8_unpack(B.q8_plan(N, H, B.MOE_BF16), q, s)), want)


def test_pack_of_special_values():
    """Ties, the largest of a block on the border between two scales, subnormal and huge values, infinities and NaN."""
    x = torch.zeros(12, 200)
    x[1, :8] = torch.tensor([448.0, 1.0625, 1.1875, -1.0625, 2.0 ** -7 * 1.5, 2.0 ** -10, 3 * 2.0 ** -10, 17.0])
    x[2, 0], x[3, 0] = 448.0, 448.00003
    x[4, 0], x[5, 0] = 3.3e38, 1e-38
    x[6, 130] = 1e-45
    x[7, 3], x[7, 4], x[7, 5], x[7, 150] = float("inf"), float("nan"), 5.0, -float("inf")
    x[8, :] = float("nan")
    x[9, 1], x[9, 2] = -448.0 * 2.0 ** -90, 2.0 ** -99 * 1.0625
    x[10, 0], x[10, 1] = 1.75, 1.7500001
    x = x.to(DEV)
    plan = B.q8_plan(12, 200, B.MOE_F32)
    q, s = B.q8_pack(plan, x)
    back = B.q8_unpack(plan, q, s)
    want, e = Q.quantise(dev_to_f64(x))
    got, _, ge = values8(q, s, 200)
    assert np.array_equal(ge, e) and np.array_equal(got, want, equal_nan=True)
    # 3.3e38 = 248.3 * 2^120 lies nearest to 256 * 2^120 = 2^128, which fp32 does not hold
    assert want[4, 0] == 2.0 ** 128
    with np.errstate(over="ignore"):
        assert np.array_equal(back.cpu().numpy(), want.astype(np.float32), equal_nan=True)


def test_unpack_of_every_byte():
    """All e4m3 codes under all scales: the value where fp32 holds it, NaN for NaN on either side."""
    q = torch.arange(256, dtype=torch.uint8).repeat(256, 1)
    s = torch.full((256, 4), 127, dtype=torch.uint8)
    s[:, 0] = s[:, 1] = torch.arange(256, dtype=torch.uint8)
    back = B.q8_unpack(B.q8_plan(256, 256, B.MOE_F32), q.view(B.E4M3).to(DEV), s.view(B.E8M0).to(DEV))
    scale = 2.0 ** (np.arange(256.0) - 127)[:, None]
    scale[255] = np.nan
    with np.errstate(over="ignore"):
        want = (Q.decode(q.numpy()) * scale).astype(np.float32)
    assert np.array_equal(back.cpu().numpy(), want, equal_nan=True)


@pytest.mark.parametrize("dtype", sorted(TYPES))
@pytest.mark.parametrize("shape", [(1, 1, 1), (2, 128, 128), (3, 130, 72), (1, 1000, 264), (2, 5, 300), (1, 257, 513), (5, 64, 640)], ids=str)
def test_pack_weights(shape, dtype):
    E, K, N = shape
    w = rows(E * K, N, dtype, spread=0.5).view(E, K, N)
    qt, st, q, s = B.q8_pack_weights(w)
    only = B.q8_pack_weights(w, "K"), B.q8_pack_weights(w, "N")
    torch.cuda.synchronize()
    for a, b in zip((qt, st, q, s), (*only[0], *only[1])):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    want, e = Q.quantise_weights(dev_to_f64(w))
    n = lambda t: t.view(torch.uint8).cpu().numpy()
    kb, nb = -(-K // 128), -(-N // 128)
    assert np.array_equal(n(s)[:, :, :nb].astype(int) - 127, e) and np.all(n(s)[:, :, nb:] == 127)
    assert np.array_equal(n(st)[:, :, :kb].astype(int) - 127, e.transpose(0, 2, 1)) and np.all(n(st)[:, :, kb:] == 127)
    full = np.repeat(np.repeat(2.0 ** e, 128, 1), 128, 2)[:, :K, :N]
    assert np.array_equal(Q.decode(n(q)[:, :, :N]) * full, want) and np.all(n(q)[:, :, N:] & 127 == 0)
    assert np.array_equal(Q.decode(n(qt)[:, :, :K]) * full.transpose(0, 2, 1), want.transpose(0, 2, 1)) and np.all(n(qt)[:, :, K:] & 127 == 0)


def swiglu_inputs(N, H, dtype, seed=1):
    a, u, dh = rows(N, H, dtype, seed, 0.5), rows(N, H, dtype, seed + 1, 0.5), rows(N, H, dtype, seed + 2, 0.5)
    if H > 6:
        a[0, :6] = torch.tensor([0.0, -0.0, 60.0, -60.0, -95.0, -300.0])
    return a, u, dh


@pytest.mark.parametrize("dtype", sorted(TYPES))
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "%dx%d" % s)
def test_swiglu(size, dtype):
    require_lib()
    N, H = size
    a, u, dh = swiglu_inputs(max(N, 1), H, dtype)
    a, u, dh = a[:N], u[:N], dh[:N]
    e = TYPES[dtype][1]
    plan = B.q8_plan(N, H, B.moe_dtype(a.dtype))
    hq, hs, kept = B.q8_swiglu_forward(plan, a, u)
    hq2, hs2, none = B.q8_swiglu_forward(plan, a, u, keep=False)
    dA, dU = B.q8_swiglu_backward(plan, kept, dh)
    over = dh.clone()
    dA2, dU2 = B.q8_swiglu_backward(plan, kept, over, dA=over)
    torch.cuda.synchronize()
    if N == 0:
        return
    assert none is None and torch.equal(dA, dA2) and torch.equal(dU, dU2)
    assert torch.equal(hq.view(torch.uint8), hq2.view(torch.uint8)) and torch.equal(hs.view(torch.uint8), hs2.view(torch.uint8))
    a64, u64, d64 = dev_to_f64(a), dev_to_f64(u), dev_to_f64(dh)
    with np.errstate(over="ignore"):
        h = Q.swiglu(a64, u64)
    check8(hq, hs, h, (8 + np.abs(a64)) * U * np.abs(h) + 2.0 ** -120)
    for pair, x in ((kept[:2], a), (kept[2:], u)):
        want, se = Q.quantise(dev_to_f64(x))
        got, _, ge = values8(*pair, H)
        assert np.array_equal(got, want) and np.array_equal(ge, se)
    a64, u64 = values8(*kept[:2], H)[0], values8(*kept[2:], H)[0]
    with np.errstate(over="ignore"):
        ra, ru = Q.swiglu_backward(a64, u64, d64)
        g = 1 / (1 + np.exp(-a64))
    t = np.abs(a64)
    tol = np.abs(d64 * u64 * g) * ((t * (6 + t) + 4) + (8 + t) * np.abs(1 + a64 * (1 - g))) * U + 2.0 ** -120
    assert np.all(np.abs(dev_to_f64(dA) - ra) <= tol * (1 + e) + e * np.abs(ra)), "dA"
    assert np.all(np.abs(dev_to_f64(dU) - ru) <= (8 + t) * U * np.abs(ru) * (1 + e) + 2.0 ** -120 + e * np.abs(ru)), "dU"


def test_swiglu_bad_values_spoil_their_place_alone():
    a, u, dh = swiglu_inputs(8, 300, "bf16")
    plan = B.q8_plan(8, 300)
    good = B.q8_swiglu_forward(plan, a, u)
    a[3, 20], u[5, 200] = float("nan"), float("inf")
    hq, hs, kept = B.q8_swiglu_forward(plan, a, u)
    for (x, y) in ((hq, good[0]), (kept[0], good[2][0]), (kept[2], good[2][2])):
        x, y = x.view(torch.uint8), y.view(torch.uint8)
        assert torch.equal(x[[0, 1, 2, 4, 6, 7]], y[[0, 1, 2, 4, 6, 7]])
    assert torch.isnan(hq.float()[3, 20]) and torch.isnan(kept[0].float()[3, 20]) and torch.isnan(kept[2].float()[5, 200])
    assert int(torch.isnan(hq.float()).sum()) == 2


def test_blocks_past_32_bits():
    """More than 2^31 values: the last rows are as in a call of their own."""
    N, H = 600_000, 4096
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB")
    x = torch.randn(64, H, device=DEV).bfloat16().repeat(N // 64, 1)
    q, s = B.q8_pack(B.q8_plan(N, H), x)
    q2, s2 = B.q8_pack(B.q8_plan(32, H), x[-32:].contiguous())
    assert torch.equal(q[-32:].view(torch.uint8), q2.view(torch.uint8)) and torch.equal(s[-32:].view(torch.uint8), s2.view(torch.uint8))
    del x
    back = B.q8_unpack(B.q8_plan(N, H), q, s)
    assert torch.equal(back[-32:], B.q8_unpack(B.q8_plan(32, H), q2, s2))


def test_fp32_swiglu_is_rounded_once():
    """Values next to where e4m3 or a scale turn are formed in 64 bits: all numbers and scales are those of the fp64 h."""
    require_lib()
    N, H = 2000, 1500
    a, u = rows(N, H, "f32", 5, 0.5), rows(N, H, "f32", 6, 0.5)
    a[3], u[4], a[5], u[5] = 0.0, -0.0, -200.0, 1e30
    hq, hs, _ = B.q8_swiglu_forward(B.q8_plan(N, H, B.MOE_F32), a, u)
    want, e = Q.quantise(Q.swiglu(dev_to_f64(a), dev_to_f64(u)))
    got, _, ge = values8(hq, hs, H)
    assert np.array_equal(got, want) and np.array_equal(ge, e)


def all_classes():
    """a [N][1] and u [1][128] of every bfloat16 mantissa: a of both signs with 2^-9 <= |a| < 2^7, u in [1, 2)."""
    a = (torch.arange(118 << 7, 134 << 7, dtype=torch.int32) << 16).view(torch.float32)
    u = (((127 << 7) | torch.arange(128, dtype=torch.int32)) << 16).view(torch.float32)
    return torch.cat([a, -a])[:, None], u[None]


@pytest.mark.parametrize("dtype", sorted(TYPES))
def test_swiglu_of_every_mantissa_is_rounded_once(dtype):
    """h next to where e4m3 turns is formed in 64 bits in bfloat16 too: from a = 17 on silu(a) is a to within fp32, so that
    a u, which may be a tie, stands for an h below it; for other a the 32-bit h is off by its exponential's argument.  All
    numbers and scales are those of the fp64 h."""
    require_lib()
    a, u = (t.expand(4096, 128).contiguous().to(TYPES[dtype][0]).to(DEV) for t in all_classes())
    for x, y in ((a, u), (a, -u * 2.0 ** -20), (a[:, :1].expand(-1, 128).contiguous(), u[:, :1] * torch.exp2(torch.arange(128.0, device=DEV) - 64).to(u.dtype))):
        hq, hs, _ = B.q8_swiglu_forward(B.q8_plan(4096, 128, B.moe_dtype(a.dtype)), x, y.contiguous())
        want, e = Q.quantise(Q.swiglu(dev_to_f64(x), dev_to_f64(y)))
        got, _, ge = values8(hq, hs, 128)
        assert int((got != want).sum()) == 0 and np.array_equal(ge, e)


@pytest.mark.parametrize("H", [1536, 1000])
def test_bf16_swiglu_is_rounded_once(H):
    """As test_fp32_swiglu_is_rounded_once, of ordinary rows, with ones whose gates are all past 17."""
    a, u = rows(2000, H, "bf16", 5, 0.5), rows(2000, H, "bf16", 6, 0.5)
    a[:40] = (a[:40].abs() + 17).bfloat16()
    a[50], u[51], a[52], u[52] = 0.0, -0.0, -200.0, 1e30
    hq, hs, _ = B.q8_swiglu_forward(B.q8_plan(2000, H), a, u)
    want, e = Q.quantise(Q.swiglu(dev_to_f64(a), dev_to_f64(u)))
    got, _, ge = values8(hq, hs, H)
    assert np.array_equal(got, want) and np.array_equal(ge, e)


@pytest.mark.parametrize("dtype", sorted(TYPES))
def test_swiglu_where_the_32_bit_exponential_ends(dtype):
    """Gates so far below zero that e^-a leaves fp32's range (-87.3 for its reciprocal, -88.7 for itself), under factors
    that bring the products back: h, dA and dU are those of fp64, not 0.  The gradients are rounded to fp32 and to the
    output's type: half a step of each, or of the least number."""
    require_lib()
    dt, e = TYPES[dtype]
    a = torch.tensor([-80.0, -87.0, -87.5, -88.0, -89.0, -95.0, -100.0, -104.0, -120.0, -300.0, -700.0, -800.0])[:, None].expand(-1, 300)
    n = len(a)
    for u, d in ((torch.linspace(1e30, 3e38, 300), 1.0), (torch.linspace(-3.0, 3.0, 300), 1e30), (torch.full((300,), 1e38), 1e-3)):
        x, y, dh = a.to(dt).contiguous().to(DEV), u.expand(n, -1).to(dt).contiguous().to(DEV), torch.full((n, 300), d).to(dt).to(DEV)
        plan = B.q8_plan(n, 300, B.moe_dtype(dt))
        hq, hs, kept = B.q8_swiglu_forward(plan, x, y)
        dA, dU = B.q8_swiglu_backward(plan, kept, dh)
        with np.errstate(over="ignore"):
            want, se = Q.quantise(Q.swiglu(dev_to_f64(x), dev_to_f64(y)))
            got, _, ge = values8(hq, hs, 300)
            assert np.array_equal(got, want) and np.array_equal(ge, se)
            refs = Q.swiglu_backward(values8(*kept[:2], 300)[0], values8(*kept[2:], 300)[0], dev_to_f64(dh))
        far = dev_to_f64(x) < -87
        for t, ref in zip((dA, dU), refs):
            tol = (e + 2 * U) * np.abs(ref) + (2.0 ** -134 if dtype == "bf16" else 2.0 ** -150)
            assert np.all(np.abs(dev_to_f64(t) - ref)[far] <= tol[far])


def test_rows_past_one_launch():
    """More blocks than a launch has (2^29 - 32, HIP's 2^32 threads): the rows of the second are as those of the first."""
    require_lib()
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 140 << 30:
        pytest.skip("needs 140 GB")
    H, n = 8, 1 << 16
    N = (1 << 29) + n
    x = torch.randn(n, H, device=DEV).bfloat16()
    X, few, many = x.repeat(N // n, 1), B.q8_plan(n, H), B.q8_plan(N, H)
    raw = lambda t: t.view(torch.uint8)

    def same(q, s, q1, s1):
        for part in (slice(0, n), slice(N - 2 * n, N - n), slice(N - n, N)):
            assert torch.equal(raw(q)[part], raw(q1)) and torch.equal(raw(s)[part], raw(s1))

    q, s = B.q8_pack(many, X)
    q1, s1 = B.q8_pack(few, x)
    same(q, s, q1, s1)
    back = B.q8_unpack(many, q, s)
    assert bool((back.view(-1, n, H) == B.q8_unpack(few, q1, s1)).all())
    dA, dU = B.q8_swiglu_backward(many, (q, s, q, s), X, dA=X, dU=back)
    dA1, dU1 = B.q8_swiglu_backward(few, (q1, s1, q1, s1), x)
    assert bool((dA.view(-1, n, H) == dA1).all()) and bool((dU.view(-1, n, H) == dU1).all())
    del back, dU
    X.copy_(x.repeat(N // n, 1))
    B.q8_swiglu_forward(many, X, X, keep=False, H=(q, s))
    same(q, s, *B.q8_swiglu_forward(few, x, x, keep=False)[:2])
    del q, s, X, dA
    torch.cuda.empty_cache()
