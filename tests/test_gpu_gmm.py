"""Products grouped by expert on the GPU against fp64 on the same inputs.

A sum of n products in fp32 is off by at most 2 u per addition of the sum of its terms' sizes, u = 2^-24 (a whole step,
since the matrix unit need not round its inner additions to nearest): 2 u n S.  The products of bfloat16 numbers, and
those of e4m3 numbers times powers of two, are exact.  Y and dX are rounded once: 2^-8.  With accumulate, one more
addition: u of the result.

gmm8_forward multiplies e4m3 numbers with the matrix instruction for them, which adds eight products at a time before
they reach the fp32 accumulator, each cut where it lies 2^13 below the largest of the eight (measured: 2^16 - 2^16 + t
of one eight keeps t from 2^3 on, of different eights from 2^-7 on).  The seven others lose less than 2^-13 of the
largest each, so a sum loses less than 7 * 2^-13 S: TRUNC S below.  Cuts of many products do not all go one way, so
over a whole matrix the 2-norm of the error stays under 2^-13 of S's beside the output's rounding."""

import numpy as np
import pytest
import torch

from gpu_common import DEV, B, needs_gpu, require_lib
from oracle import q8_oracle as Q

pytestmark = [pytest.mark.gpu, needs_gpu]
U, E16 = 2.0 ** -24, 2.0 ** -8
TRUNC = 7 * 2.0 ** -13


def ragged(R, E, seed, skew=0.7):
    g = torch.Generator().manual_seed(seed)
    share = torch.arange(1, E + 1).double().pow(-skew)[torch.randperm(E, generator=g)]
    return torch.bincount(torch.multinomial(share, R, True, generator=g), minlength=E).tolist() if R else [0] * E


def offsets_of(sizes, start=0):
    return torch.tensor([start] + (start + np.cumsum(sizes)).tolist(), dtype=torch.int32, device=DEV)


def normal(g, *shape, std=1.0):
    return (torch.randn(*shape, generator=g) * std).bfloat16().to(DEV)


def by_expert(offsets):
    o = offsets.tolist()
    return [(e, slice(o[e], o[e + 1])) for e in range(len(o) - 1)]


def close(got, ref, size, n, e, what, cut=0.0):
    got = got.double()
    bad = (got - ref).abs() > (2 * U * max(n, 1) + cut) * size * (1 + e) + e * ref.abs()
    assert not bad.any(), (what, int(bad.sum()), float((got - ref).abs().max()))
    if cut and len(ref):
        assert float((got - ref).norm()) <= e * float(ref.norm()) + 2.0 ** -13 * float(size.norm()), what


def check_bf16(R, K, N, sizes, seed=0, start=0, after=0, offsets="given"):
    """Forward, dX, dW with `start` rows before the first expert's and `after` rows behind the last's."""
    g = torch.Generator().manual_seed(seed)
    E, R = len(sizes), sum(sizes) + start + after
    X, dY, W = normal(g, R, K), normal(g, R, N), normal(g, E, K, N, std=0.05)
    off = offsets_of(sizes, start) if offsets == "given" else None
    plan = B.gmm_plan(R, K, N, E)
    sentinel = lambda *s: torch.full(s, 77.0, dtype=torch.bfloat16, device=DEV)
    Y = B.gmm_forward(plan, X, W, off, Y=sentinel(R, N))
    dX = B.gmm_backward_dx(plan, dY, W, off, dX=sentinel(R, K))
    dW = B.gmm_backward_dw(plan, X, dY, off, dW=torch.full((E, K, N), float("nan"), device=DEV))
    old = torch.randn(E, K, N, generator=g).to(DEV)
    more = B.gmm_backward_dw(plan, X, dY, off, dW=old.clone(), accumulate=True)
    torch.cuda.synchronize()
    for e, r in by_expert(off if off is not None else offsets_of(sizes)):
        x, d, w = X[r].double(), dY[r].double(), W[e].double()
        close(Y[r], x @ w, x.abs() @ w.abs(), K, E16, ("Y", e))
        close(dX[r], d @ w.T.contiguous(), d.abs() @ w.abs().T.contiguous(), N, E16, ("dX", e))
        xt = x.T.contiguous()
        ref, size, n = xt @ d, xt.abs() @ d.abs(), r.stop - r.start
        close(dW[e], ref, size, n, 0, ("dW", e))
        o = old[e].double()
        bad = (more[e].double() - o - ref).abs() > 2 * U * n * size + U * ((o + ref).abs() + 2 * U * n * size)
        assert not bad.any(), ("accumulate", e)
        if n == 0:
            assert not dW[e].any() and torch.equal(more[e], old[e])
    for t in (Y, dX):
        assert bool((t[:start] == 77).all()) and bool((t[R - after:] == 77).all() if after else True)


def rows8(g, R, K):
    """8-bit rows of their own scales: bytes as q8_pack writes them, and their values in fp64."""
    x = torch.randn(R, K, generator=g) * torch.exp(torch.randn(R, 1, generator=g))
    plan = B.q8_plan(R, K, B.MOE_F32)
    q, s = B.q8_pack(plan, x.to(DEV))
    return q, s, B.q8_unpack(plan, q, s).double()


def check_q8(R, K, N, sizes, seed=0, start=0, after=0):
    g = torch.Generator().manual_seed(seed)
    E, R = len(sizes), sum(sizes) + start + after
    Xq, Xs, X = rows8(g, R, K)
    W = (torch.randn(E, K, N, generator=g) * 0.05 * torch.exp(torch.randn(1, 1, N, generator=g))).to(DEV)
    Wq, Ws = B.q8_pack_weights(W, "K")
    # the packed weights' values
    nb, kb = -(-N // 128), -(-K // 128)
    s = torch.exp2(Ws.view(torch.uint8)[:, :, :kb].double() - 127)
    Wv = Wq[:, :, :K].double() * s.repeat_interleave(128, 1)[:, :N].repeat_interleave(128, 2)[:, :, :K]
    off = offsets_of(sizes, start)
    dY = normal(g, R, N)
    plan = B.gmm_plan(R, K, N, E, B.GMM_Q8)
    Y = B.gmm8_forward(plan, Xq, Xs, Wq, Ws, off, Y=torch.full((R, N), 77.0, dtype=torch.bfloat16, device=DEV))
    dW = B.gmm8_backward_dw(plan, Xq, Xs, dY, off, dW=torch.full((E, K, N), float("nan"), device=DEV))
    old = torch.randn(E, K, N, generator=g).to(DEV)
    more = B.gmm8_backward_dw(plan, Xq, Xs, dY, off, dW=old.clone(), accumulate=True)
    torch.cuda.synchronize()
    assert nb == Ws.shape[1]
    for e, r in by_expert(off):
        x, d, w = X[r], dY[r].double(), Wv[e].T.contiguous()
        close(Y[r], x @ w, x.abs() @ w.abs(), K, E16, ("Y", e), TRUNC)
        xt = x.T.contiguous()
        ref, size, n = xt @ d, xt.abs() @ d.abs(), r.stop - r.start
        close(dW[e], ref, size, n, 0, ("dW", e))
        o = old[e].double()
        bad = (more[e].double() - o - ref).abs() > 2 * U * n * size + U * ((o + ref).abs() + 2 * U * n * size)
        assert not bad.any(), ("accumulate", e)
    assert bool((Y[:start] == 77).all()) and bool((Y[R - after:] == 77).all() if after else True)


# (K, N, rows of each expert): one row, one expert, empty ones first, last and between, tiles' borders, odd sizes
CASES = [
    (8, 8, [1]), (64, 64, [64]), (128, 128, [128, 0, 256]), (520, 264, ragged(1000, 7, 3, 1.5)), (72, 200, [0, 3, 0, 0, 129, 1, 0]),
    (256, 512, [257, 255, 1]), (1024, 136, [16]), (2048, 1408, [2, 0, 1, 3, 1, 0, 0, 4]), (264, 1000, [33, 31, 32, 64, 65, 63]),
    (4096, 256, [5]), (16, 2048, [300]), (8, 520, [1, 1, 1, 1]), (640, 8, [77, 500]), (136, 72, ragged(3000, 70, 4)), (384, 384, ragged(700, 130, 5)),
    (1408, 512, [1000, 24]), (512, 768, [513, 511]), (96, 96, [2000]), (7168, 256, [3]), (256, 7168, [2, 2]),
]


@pytest.mark.parametrize("K,N,sizes", CASES, ids=lambda v: str(v) if isinstance(v, int) else "E%d_R%d" % (len(v), sum(v)))
def test_bf16(K, N, sizes):
    require_lib()
    check_bf16(0, K, N, sizes)


@pytest.mark.parametrize("K,N,sizes", [(K - d, N, s) for (K, N, s), d in zip(CASES, [0, 1, 0, 7, 3, 0, 127, 0, 100, 0, 15, 7, 0, 5, 1, 0, 0, 1, 0, 0])],
                         ids=lambda v: str(v) if isinstance(v, int) else "E%d_R%d" % (len(v), sum(v)))
def test_q8(K, N, sizes):
    require_lib()
    check_q8(0, K, N, sizes)


# (K, N, rows): every tile that a product can take, with tiles that end inside a matrix and inside an expert, and the
# splits of k: over few tiles, into parts of which the last is shorter, and of an expert's rows
TILES = [
    (136, 4104, ragged(3000, 3, 10, 0.3)), (4104, 136, ragged(3000, 3, 11, 0.3)),  # 256 x 256
    (200, 1032, ragged(2800, 40, 12, 0.1)), (1032, 200, ragged(2800, 40, 13, 0.1)),  # 128 x 128
    (200, 1032, ragged(1300, 40, 14, 0.4)), (1032, 200, ragged(1300, 40, 15, 0.4)),  # 64 x 128
    (200, 1032, ragged(500, 64, 16)), (1032, 200, ragged(500, 64, 17)),  # 16 or 32 x 128
    (520, 520, ragged(900, 40, 18)),  # dW in 256 x 256
    (2056, 72, [70]), (72, 2056, [70]), (5000, 136, [3, 0, 9]), (72, 64, [5000]), (64, 200, [3000, 0, 40, 1])]


@pytest.mark.parametrize("check", [check_bf16, check_q8])
@pytest.mark.parametrize("K,N,sizes", TILES, ids=lambda v: str(v) if isinstance(v, int) else "E%d_R%d" % (len(v), sum(v)))
def test_every_tile_and_split(check, K, N, sizes):
    check(0, K, N, sizes)


# experts of more than twice the mean rows, which go first in dW, among others, in every set of 64 experts, with even and
# odd counts of tiles along both
def hot(E, where, rows=400):
    sizes = ragged(2 * E, E, 21, 0.3)
    for e in where:
        sizes[e] += rows
    return sizes


HOT = [(520, 264, hot(70, [0, 3, 63, 64, 69])), (1288, 648, hot(10, [9])), (264, 72, hot(300, [17, 128, 255, 256, 299], 90)),
       (72, 136, hot(1024, [5, 600, 1023], 300)), (136, 200, hot(3, [2], 2000))]


@pytest.mark.parametrize("check", [check_bf16, check_q8])
@pytest.mark.parametrize("K,N,sizes", HOT, ids=lambda v: str(v) if isinstance(v, int) else "E%d_R%d" % (len(v), sum(v)))
def test_large_experts_among_others(check, K, N, sizes):
    check(0, K, N, sizes)


# one to four rows: K on both sides of a KiB and of its multiples, more experts than rows, rows of no expert
SINGLE = [(1, 8, [1]), (100, 72, [1, 0, 1]), (128, 264, [0, 2]), (1000, 136, [1]), (1024, 136, [3]), (1025, 24, [1, 1, 1, 1]),
          (2049, 72, [0, 0, 4, 0]), (4096, 264, [2]), (4097, 136, [1, 2]), (7168, 520, [1]), (10000, 40, [0] * 200 + [1, 0, 2])]


@pytest.mark.parametrize("start,after", [(0, 0), (1, 0), (0, 1)])
@pytest.mark.parametrize("K,N,sizes", SINGLE, ids=lambda v: str(v) if isinstance(v, int) else "E%d_R%d" % (len(v), sum(v)))
def test_few_rows_in_8_bits(K, N, sizes, start, after):
    if sum(sizes) + start + after > 4:
        sizes = [min(n, 1) for n in sizes]
    check_q8(0, K, N, sizes, start=start, after=after)


def test_splits_are_taken():
    """The cases above reach the joins of partial sums."""
    assert B.gmm_plan(70, 2056, 72, 1).fwd_workspace_bytes > 0 and B.gmm_plan(70, 72, 2056, 1).fwd_workspace_bytes > 0
    assert B.gmm_plan(12, 5000, 136, 3, B.GMM_Q8).fwd_workspace_bytes > 0
    assert B.gmm_plan(5000, 72, 64, 1).bwd_workspace_bytes > 0 and B.gmm_plan(3041, 64, 200, 4).bwd_workspace_bytes > 0


@pytest.mark.parametrize("check", [check_bf16, check_q8])
def test_rows_of_no_expert_are_left(check):
    check(0, 136, 136, [40, 0, 100, 7], start=13, after=200)
    check(0, 136, 264, [0, 0, 0], start=5, after=9)
    check(0, 264, 136, [300], start=1, after=1)
    check(0, 4096, 136, [5, 0, 6], start=3, after=2)
    check(0, 72, 64, [2000, 0, 900], start=300, after=100)


def test_without_offsets():
    check_bf16(0, 264, 392, [530], offsets="none")
    g = torch.Generator().manual_seed(1)
    q, s, _ = rows8(g, 530, 300)
    Wq, Ws = B.q8_pack_weights(torch.randn(1, 300, 264, generator=g).to(DEV), "K")
    plan = B.gmm_plan(530, 300, 264, 1, B.GMM_Q8)
    dY = normal(g, 530, 264)
    off = offsets_of([530])
    assert torch.equal(B.gmm8_forward(plan, q, s, Wq, Ws), B.gmm8_forward(plan, q, s, Wq, Ws, off))
    assert torch.equal(B.gmm8_backward_dw(plan, q, s, dY), B.gmm8_backward_dw(plan, q, s, dY, off))


def test_all_experts_of_a_large_count():
    check_bf16(0, 64, 72, ragged(2500, 1024, 9, 0.3))
    check_q8(0, 130, 64, ragged(2500, 1000, 9, 0.3))


def test_no_rows():
    W, off = torch.randn(2, 16, 8, device=DEV).bfloat16(), offsets_of([0, 0])
    x, dy = torch.empty(0, 16, dtype=torch.bfloat16, device=DEV), torch.empty(0, 8, dtype=torch.bfloat16, device=DEV)
    plan = B.gmm_plan(0, 16, 8, 2)
    assert B.gmm_forward(plan, x, W, off).numel() == 0 and B.gmm_backward_dx(plan, dy, W, off).numel() == 0
    assert not B.gmm_backward_dw(plan, x, dy, off, dW=torch.ones(2, 16, 8, device=DEV)).any()
    old = torch.ones(2, 16, 8, device=DEV)
    assert bool((B.gmm_backward_dw(plan, x, dy, off, dW=old, accumulate=True) == 1).all())


@pytest.mark.parametrize("q8", [False, True])
def test_bad_rows_spoil_their_expert_alone(q8):
    """NaN in rows of one expert, and in rows of none: the neighbours' outputs are bit for bit as without."""
    sizes, K, N = [50, 70, 0, 90], 136, 264
    g = torch.Generator().manual_seed(2)
    R = sum(sizes) + 30
    X, dY, W = normal(g, R, K), normal(g, R, N), normal(g, 4, K, N)
    off = offsets_of(sizes, 10)
    plan = B.gmm_plan(R, K, N, 4, B.GMM_Q8 if q8 else B.GMM_BF16)
    rp = B.q8_plan(R, K)
    Wq, Ws = B.q8_pack_weights(W, "K")

    def run():
        if q8:
            Xq, Xs = B.q8_pack(rp, X)
            return B.gmm8_forward(plan, Xq, Xs, Wq, Ws, off), None, B.gmm8_backward_dw(plan, Xq, Xs, dY, off)
        return B.gmm_forward(plan, X, W, off), B.gmm_backward_dx(plan, dY, W, off), B.gmm_backward_dw(plan, X, dY, off)

    good = run()
    for t in (X, dY):
        t[:10] = float("nan")
        t[-20:] = float("inf")
        t[10 + 60] = float("nan")  # expert 1
    bad = run()
    rows = [r for r in range(10, R - 20) if r != 70]
    for a, b in zip(good[:2], bad[:2]):
        if a is not None:
            assert torch.equal(a[rows], b[rows]) and torch.isnan(b[70]).all()
    assert torch.equal(good[2][[0, 2, 3]], bad[2][[0, 2, 3]]) and torch.isnan(bad[2][1]).all()


@pytest.mark.parametrize("K,N", [(136, 264), (200, 72), (64, 1032)])
@pytest.mark.parametrize("q8", [False, True])
def test_a_bad_matrix_spoils_its_expert_alone(q8, K, N):
    """NaN and infinities in one expert's W: tiles and steps that end inside a matrix read nothing of the next."""
    sizes = [60, 70, 0, 90]
    g = torch.Generator().manual_seed(7)
    X, dY, W, off = normal(g, 220, K), normal(g, 220, N), normal(g, 4, K, N), offsets_of(sizes)
    plan = B.gmm_plan(220, K, N, 4, B.GMM_Q8 if q8 else B.GMM_BF16)

    def run():
        if q8:
            return [B.gmm8_forward(plan, *B.q8_pack(B.q8_plan(220, K), X), *B.q8_pack_weights(W, "K"), off)]
        return [B.gmm_forward(plan, X, W, off), B.gmm_backward_dx(plan, dY, W, off)]

    good = run()
    W[1], W[2] = float("nan"), float("inf")  # (expert 2 has no rows)
    for a, b in zip(good, run()):
        assert torch.equal(a[:60], b[:60]) and torch.equal(a[130:], b[130:]) and torch.isnan(b[60:130]).all()


def test_scale_bytes_at_their_ends():
    """NaN's byte makes its row (in dW its block of columns) NaN and nothing else; the least and largest scales hold."""
    R, K, N = 40, 300, 136
    g = torch.Generator().manual_seed(8)
    q, s, _ = rows8(g, R, K)
    W = torch.randn(1, K, N, generator=g).to(DEV)
    Wq, Ws = B.q8_pack_weights(W, "K")
    dY = normal(g, R, N)
    plan = B.gmm_plan(R, K, N, 1, B.GMM_Q8)
    good, dgood = B.gmm8_forward(plan, q, s, Wq, Ws), B.gmm8_backward_dw(plan, q, s, dY)
    b = s.view(torch.uint8)
    b[7, 1] = 255
    y, dw = B.gmm8_forward(plan, q, s, Wq, Ws), B.gmm8_backward_dw(plan, q, s, dY)
    rows = [r for r in range(R) if r != 7]
    assert torch.equal(y[rows], good[rows]) and torch.isnan(y[7]).all()
    assert torch.isnan(dw[0, 128:256]).all() and torch.equal(dw[0, :128], dgood[0, :128]) and torch.equal(dw[0, 256:], dgood[0, 256:])
    for byte in (17, 0, 237):  # 2^-110; 2^-127, whose values no longer show; 2^110
        b[:] = byte
        x = q.double()[:, :K] * 2.0 ** (byte - 127)
        w = (Wq[0, :, :K].double() * torch.exp2(Ws.view(torch.uint8)[0, :, :3].double() - 127).repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]).T.contiguous()
        ref, size = x @ w, x.abs() @ w.abs()
        tiny = 2.0 ** -126 if byte == 0 else 0.0  # what underflows in fp32
        got = B.gmm8_forward(plan, q, s, Wq, Ws).double()
        assert not ((got - ref).abs() > (2 * U * K + TRUNC) * size * (1 + E16) + E16 * ref.abs() + tiny).any(), byte


def test_few_rows_with_bad_values():
    """The product of few rows: NaN in a row or its scale, and in another expert's matrix, stay there; the least and
    largest scales hold; the same bits on every pass and whatever the other rows are."""
    R, K, N = 4, 1300, 136
    g = torch.Generator().manual_seed(9)
    q, s, _ = rows8(g, R, K)
    W = torch.randn(3, K, N, generator=g).to(DEV)
    Wq, Ws = B.q8_pack_weights(W, "K")
    off = offsets_of([1, 0, 3])
    plan = B.gmm_plan(R, K, N, 3, B.GMM_Q8)
    good = B.gmm8_forward(plan, q, s, Wq, Ws, off)
    Wq2 = Wq.clone().view(torch.uint8)
    Wq2[0, 5, 1290], Wq2[1] = 127, 127  # NaN in expert 0's column 5, and all over expert 1, which has no rows
    q2, s2 = q.clone().view(torch.uint8), s.clone().view(torch.uint8)
    q2[2, 1299], s2[3, 10] = 127, 255
    got = B.gmm8_forward(plan, q2.view(q.dtype), s2.view(s.dtype), Wq2.view(Wq.dtype), Ws, off)
    assert torch.isnan(got[0, 5]) and torch.isnan(got[2:]).all()
    keep = [n for n in range(N) if n != 5]
    assert torch.equal(got[0, keep], good[0, keep]) and torch.equal(got[1], good[1])
    wb = Ws.view(torch.uint8)[:, :, :11].double() - 127
    w = Wq[:, :, :K].double() * torch.exp2(wb).repeat_interleave(128, 1)[:, :N].repeat_interleave(128, 2)[:, :, :K]
    for byte in (17, 0, 237):
        s2[:] = byte
        got = B.gmm8_forward(plan, q, s2.view(s.dtype), Wq, Ws, off).double()
        x = q.double()[:, :K] * 2.0 ** (byte - 127)
        for r, e in enumerate((0, 2, 2, 2)):
            ref, size = w[e] @ x[r], w[e].abs() @ x[r].abs()
            tiny = 2.0 ** -126 if byte == 0 else 0.0  # what underflows in fp32
            assert not ((got[r] - ref).abs() > 2 * U * K * size * (1 + E16) + E16 * ref.abs() + tiny).any(), (byte, r)


def test_matrices_past_32_bits():
    """More than 2^31 values in X, dY and dX: the last expert's rows and matrix."""
    R, K, N = 270_000, 8192, 64
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    g = torch.Generator().manual_seed(9)
    part = normal(g, 1000, K)
    X = part.repeat(R // 1000, 1)
    W, dY, off = normal(g, 2, K, N, std=0.05), normal(g, 1000, N).repeat(R // 1000, 1), offsets_of([R - 700, 700])
    plan = B.gmm_plan(R, K, N, 2)
    last = slice(R - 700, R)
    x, d, w = X[last].double(), dY[last].double(), W[1].double()
    close(B.gmm_forward(plan, X, W, off)[last], x @ w, x.abs() @ w.abs(), K, E16, "Y")
    dX = B.gmm_backward_dx(plan, dY, W, off)
    close(dX[last], d @ w.T.contiguous(), d.abs() @ w.abs().T.contiguous(), N, E16, "dX")
    del dX
    dW = B.gmm_backward_dw(plan, X, dY, off)
    xt = x.T.contiguous()
    close(dW[1], xt @ d, xt.abs() @ d.abs(), 700, 0, "dW")
    Xq, Xs = B.q8_pack(B.q8_plan(R, K), X)
    del X
    plan = B.gmm_plan(R, K, N, 2, B.GMM_Q8)
    Wq, Ws = B.q8_pack_weights(W, "K")
    xv = B.q8_unpack(B.q8_plan(700, K), Xq[last].contiguous(), Xs[last].contiguous()).double()
    s8 = torch.exp2(Ws.view(torch.uint8)[1, :, :64].double() - 127).repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)
    w = (Wq[1].double() * s8).T.contiguous()
    close(B.gmm8_forward(plan, Xq, Xs, Wq, Ws, off)[last], xv @ w, xv.abs() @ w.abs(), K, E16, "Y", TRUNC)
    xt = xv.T.contiguous()
    close(B.gmm8_backward_dw(plan, Xq, Xs, dY, off)[1], xt @ d, xt.abs() @ d.abs(), 700, 0, "dW")


@pytest.mark.parametrize("rows", [300, 3, 4000])
@pytest.mark.parametrize("operands", [B.GMM_BF16, B.GMM_Q8])
def test_broken_offsets_stay_inside(operands, rows):
    """Descending, negative and far too large offsets: whatever the rows hold, nothing around the outputs is touched."""
    R, K, N, E, pad = rows, 136, 72, 5, 4096
    g = torch.Generator().manual_seed(3)
    X, dY, W = normal(g, R, K), normal(g, R, N), normal(g, E, K, N)
    plan = B.gmm_plan(R, K, N, E, operands)
    Xq, Xs = B.q8_pack(B.q8_plan(R, K), X)
    Wq, Ws = B.q8_pack_weights(W, "K")

    def guarded(shape, dtype):
        n = int(np.prod(shape))
        buf = torch.full((n + 2 * pad,), 55.0, dtype=dtype, device=DEV)
        return buf, buf[pad:pad + n].view(shape)

    for broken in ([0, 500, 20, 300, -7, 2 ** 31 - 1], [-2 ** 31, 2 ** 31 - 1, -2 ** 31, 2 ** 31 - 1, 0, 300], [300, 200, 100, 50, 20, 0], [2 ** 31 - 1] * 6,
                   [0, 300, 0, 300, 0, 300]):
        off = torch.tensor(broken, dtype=torch.int32, device=DEV)
        (by, Y), (bx, dX), (bw, dW) = guarded((R, N), torch.bfloat16), guarded((R, K), torch.bfloat16), guarded((E, K, N), torch.float32)
        if operands == B.GMM_BF16:
            B.gmm_forward(plan, X, W, off, Y=Y)
            B.gmm_backward_dx(plan, dY, W, off, dX=dX)
            B.gmm_backward_dw(plan, X, dY, off, dW=dW)
        else:
            B.gmm8_forward(plan, Xq, Xs, Wq, Ws, off, Y=Y)
            B.gmm8_backward_dw(plan, Xq, Xs, dY, off, dW=dW)
        torch.cuda.synchronize()
        for b in (by, bx, bw):
            assert bool((b[:pad] == 55).all()) and bool((b[-pad:] == 55).all())


def test_scales_of_any_size():
    """Scales far apart between rows, blocks and columns: each enters with its own power of two."""
    g = torch.Generator().manual_seed(4)
    R, K, N = 70, 700, 264
    x = torch.randn(R, K, generator=g) * torch.exp2(torch.randint(-30, 30, (R, 1), generator=g).float())
    x = x * torch.exp2(torch.randint(-8, 8, (1, K), generator=g).float())
    plan8 = B.q8_plan(R, K, B.MOE_F32)
    Xq, Xs = B.q8_pack(plan8, x.to(DEV))
    X = B.q8_unpack(plan8, Xq, Xs).double()
    W = torch.randn(1, K, N, generator=g) * torch.exp2(torch.randint(-20, 20, (1, 1, N), generator=g).float())
    Wv = torch.from_numpy(Q.quantise_weights(W.numpy())[0])[0].to(DEV)
    Wq, Ws = B.q8_pack_weights(W.to(DEV), "K")
    Y = B.gmm8_forward(B.gmm_plan(R, K, N, 1, B.GMM_Q8), Xq, Xs, Wq, Ws)
    close(Y, X @ Wv, X.abs() @ Wv.abs(), K, E16, "Y", TRUNC)


@pytest.mark.parametrize("split", [None, (220, 4096, 72, [100, 0, 100, 20]), (4000, 72, 64, [1500, 0, 2000, 500])], ids=str)
@pytest.mark.parametrize("operands", [B.GMM_BF16, B.GMM_Q8])
def test_repeats_on_streams_and_in_graphs(operands, split):
    """Bit for bit: twice, on another stream, in two captured graphs with workspaces of their own, replayed in turn
    between eager calls, and on new inputs in the same buffers."""
    R, K, N, sizes = 700, 1000, 392, [300, 0, 250, 150]
    if split:  # k in parts, forward or over the rows
        R, K, N, sizes = split
    g = torch.Generator().manual_seed(5)
    X, dY, W, off = normal(g, R, K), normal(g, R, N), normal(g, 4, K, N), offsets_of(sizes)
    plan = B.gmm_plan(R, K, N, 4, operands)
    rp = B.q8_plan(R, K)
    Xq, Xs = B.q8_pack(rp, X)
    Wq, Ws = B.q8_pack_weights(W, "K")

    def run(ws):
        if operands == B.GMM_Q8:
            return [B.gmm8_forward(plan, Xq, Xs, Wq, Ws, off, ws=ws), B.gmm8_backward_dw(plan, Xq, Xs, dY, off, ws=ws)]
        return [B.gmm_forward(plan, X, W, off, ws=ws), B.gmm_backward_dx(plan, dY, W, off, ws=ws), B.gmm_backward_dw(plan, X, dY, off, ws=ws)]

    spaces = [B.workspace(plan, "both", DEV) for _ in range(3)]
    want = [t.clone() for t in run(spaces[0])]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = run(None)
    side.synchronize()
    assert all(map(torch.equal, want, other)) and all(map(torch.equal, want, run(None)))
    graphs = []
    for ws in spaces[1:]:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = run(ws)
        graphs.append((graph, out))
    for turn in range(3):
        if turn == 2:
            X.mul_(0.5)
            dY.copy_(dY.flip(0))
            off.copy_(offsets_of([1, R - 200, 199, 0]))
            B.q8_pack(rp, X, Xq, Xs)
            want = [t.clone() for t in run(spaces[0])]
        for graph, out in graphs:
            for t in out:
                t.fill_(9)
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert all(map(torch.equal, want, out)), turn
            run(spaces[0])


def test_gradients_are_the_adjoints():
    """<dY, X W> = <dX, X> = <dW, W>, each to the outputs' roundings."""
    g = torch.Generator().manual_seed(6)
    sizes = [100, 0, 57, 343]
    X, dY, W, off = normal(g, 500, 264), normal(g, 500, 136), normal(g, 4, 264, 136), offsets_of(sizes)
    plan = B.gmm_plan(500, 264, 136, 4)
    d = lambda a, b: float((a.double() * b.double()).sum())
    y, dx, dw = B.gmm_forward(plan, X, W, off), B.gmm_backward_dx(plan, dY, W, off), B.gmm_backward_dw(plan, X, dY, off)
    vals = d(y, dY), d(dx, X), d(dw, W)
    scale = E16 * max(float((y.double() * dY.double()).abs().sum()), float((dx.double() * X.double()).abs().sum()))
    assert max(vals) - min(vals) <= 2 * scale


# rows, K, N, experts: dot products; 64 x 64 tiles, whole and with k in parts; 32, 64 and 128 rows; 256 x 256
CUTS = [(4, 300, 72, 1), (4, 2056, 72, 2), (5, 300, 72, 1), (40, 300, 72, 1), (70, 2056, 72, 1), (500, 200, 1032, 64), (1300, 200, 1032, 40),
        (2800, 200, 1032, 40), (3000, 136, 4104, 3)]


@pytest.mark.parametrize("R,K,N,E", CUTS)
def test_8_bit_sums_that_cancel(R, K, N, E):
    """Sums whose products cancel in pairs of one eight but for small ones, under the header's bound: fp32's roundings for
    up to four rows, GMM8_CUT of the products' magnitudes beside them for more."""
    g = torch.Generator().manual_seed(11)
    x, w = torch.randn(R, K, generator=g), torch.randn(E, K, N, generator=g)
    x[:, 1::4], w[:, 1::4] = -x[:, 0::4][:, :x[:, 1::4].shape[1]], w[:, 0::4][:, :w[:, 1::4].shape[1]]
    for c in (2, 3):  # and between the pairs products of 2^-10 to 2^-15 of theirs
        x[:, c::4] *= torch.exp2(-torch.randint(10, 16, x[:, c::4].shape, generator=g).float())
    x, w = x.to(DEV), w.to(DEV)
    p8 = B.q8_plan(R, K, B.MOE_F32)
    Xq, Xs = B.q8_pack(p8, x)
    Wq, Ws = B.q8_pack_weights(w, "K")
    X = B.q8_unpack(p8, Xq, Xs).double()
    s = torch.exp2(Ws.view(torch.uint8)[:, :, :-(-K // 128)].double() - 127)
    Wv = (Wq[:, :, :K].double() * s.repeat_interleave(128, 1)[:, :N].repeat_interleave(128, 2)[:, :, :K]).transpose(1, 2).contiguous()
    sizes = ragged(R, E, 3, 0.1)
    off = offsets_of(sizes)
    Y = B.gmm8_forward(B.gmm_plan(R, K, N, E, B.GMM_Q8), Xq, Xs, Wq, Ws, off).double()
    cut = 0.0 if R <= 4 else B.GMM8_CUT
    for e, r in by_expert(off):
        ref, size = X[r] @ Wv[e], X[r].abs() @ Wv[e].abs()
        bad = (Y[r] - ref).abs() > (2 * U * K + cut) * size * (1 + E16) + E16 * ref.abs()
        assert not bad.any(), (e, int(bad.sum()))


def test_a_row_of_an_8_bit_product_does_not_depend_on_the_others():
    """In calls of the same sizes a row has the same bits whatever the other rows hold."""
    for R, K, N in ((4, 700, 136), (9, 700, 136), (200, 700, 136)):
        g = torch.Generator().manual_seed(12)
        Xq, Xs, _ = rows8(g, R, K)
        Wq, Ws = B.q8_pack_weights(torch.randn(1, K, N, generator=g).to(DEV), "K")
        plan = B.gmm_plan(R, K, N, 1, B.GMM_Q8)
        a = B.gmm8_forward(plan, Xq, Xs, Wq, Ws)
        other, scales, _ = rows8(g, R, K)
        other.view(torch.uint8)[R // 2], scales.view(torch.uint8)[R // 2] = Xq.view(torch.uint8)[R // 2], Xs.view(torch.uint8)[R // 2]
        assert torch.equal(a[R // 2], B.gmm8_forward(plan, other, scales, Wq, Ws)[R // 2])


def check_q8_dx(R, K, N, sizes, seed=0):
    """dX in 8 bits: gmm8_forward of a plan (R, N, K, E) on dY's rows in 8 bits and on W in 8 bits along N, to the bound of
    the forward product."""
    g = torch.Generator().manual_seed(seed)
    E, R = len(sizes), sum(sizes)
    Dq, Ds, D = rows8(g, R, N)
    W = (torch.randn(E, K, N, generator=g) * 0.05 * torch.exp(torch.randn(1, K, 1, generator=g)) * torch.exp(torch.randn(E, 1, N, generator=g))).to(DEV)
    Wq, Ws = B.q8_pack_weights(W, "N")
    s = torch.exp2(Ws.view(torch.uint8)[:, :, :-(-N // 128)].double() - 127)
    Wv = Wq[:, :, :N].double() * s.repeat_interleave(128, 1)[:, :K].repeat_interleave(128, 2)[:, :, :N]
    off = offsets_of(sizes)
    dX = B.gmm8_forward(B.gmm_plan(R, N, K, E, B.GMM_Q8), Dq, Ds, Wq, Ws, off)
    for e, r in by_expert(off):
        w = Wv[e].T.contiguous()
        close(dX[r], D[r] @ w, D[r].abs() @ w.abs(), N, E16, ("dX", e), 0.0 if R <= 4 else TRUNC)
        # nothing but roundings of the given W: every number within half a step of e4m3 of it
        scale = s[e].repeat_interleave(128, 0)[:K].repeat_interleave(128, 1)[:, :N]
        assert bool(((Wv[e] - W[e].double()).abs() <= torch.maximum(2.0 ** -4 * W[e].double().abs(), 2.0 ** -10 * scale)).all())


@pytest.mark.parametrize("K,N,sizes", CASES + TILES, ids=lambda v: str(v) if isinstance(v, int) else "E%d_R%d" % (len(v), sum(v)))
def test_dx_in_8_bits(K, N, sizes):
    check_q8_dx(0, K, N, sizes)
    check_q8_dx(0, K, max(N - 3, 1), sizes, 1)
