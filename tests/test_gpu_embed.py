"""Token embedding and its gradient on the GPU.

Forward: scale W[id] in fp32, rounded once: the same bits as that product.
Backward, u = 2^-24: an id's n rows are added at most 64 deep within a run's
tile and n / 16 + 8 deep across tiles, then scaled, so dW is within (64 + n /
16 + 16) u of the sum of the terms' sizes; an id that does not occur is 0."""

import numpy as np
import pytest
import torch

from gpu_common import DEV, B, dev_to_f64, needs_gpu, require_lib

pytestmark = [pytest.mark.gpu, needs_gpu]
U = 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def draw_ids(kind, N, V, r):
    if kind == "spread":
        ids = r.integers(0, V, N)
    elif kind == "skewed":
        ids = np.floor(V ** r.random(N)).astype(np.int64) - 1
    elif kind == "one":
        ids = np.full(N, V // 2)
    elif kind == "down":
        ids = np.arange(N)[::-1] % V
    else:  # padded
        ids = np.full(N, -1)
    if kind in ("spread", "skewed"):
        out = r.random(N)
        ids = np.where(out < 0.05, -1, ids)
        ids = np.where((out > 0.9) & (out < 0.92), V, ids)
        ids = np.where((out > 0.92) & (out < 0.93), 2**31 - 1, ids)
        ids = np.where((out > 0.93) & (out < 0.94), -2**31, ids)
    return ids.astype(np.int32)


def check(N, V, H, dtype, kind, scale=1.25, seed=0):
    r = np.random.default_rng(seed)
    dt = TYPES[dtype]
    ids = draw_ids(kind, N, V, r)
    g = torch.Generator().manual_seed(seed)
    W = torch.randn(V, H, generator=g).to(dt).to(DEV)
    dY = torch.randn(N, H, generator=g).to(dt).to(DEV)
    di = torch.from_numpy(ids).to(DEV)
    plan = B.embed_plan(N, V, H, B.moe_dtype(dt), scale)
    Y = B.embed_forward(plan, W, di)
    ok = (ids >= 0) & (ids < V)
    at = torch.from_numpy(np.where(ok, ids, 0).astype(np.int64)).to(DEV)
    want = torch.where(torch.from_numpy(ok).to(DEV)[:, None], W[at].float() * torch.tensor(scale, device=DEV), 0.0).to(dt)
    assert torch.equal(Y, want)
    dW = B.embed_backward(plan, di, dY)
    again = B.embed_backward(plan, di, dY)
    assert torch.equal(dW, again)
    dy = dev_to_f64(dY) * scale
    ref, size, n = np.zeros((V, H)), np.zeros((V, H)), np.bincount(ids[ok], minlength=V)[:, None]
    np.add.at(ref, ids[ok], dy[ok])
    np.add.at(size, ids[ok], np.abs(dy[ok]))
    got = dev_to_f64(dW)
    assert np.all(np.abs(got - ref) <= (64 + n / 16 + 16) * U * size)
    # onto what is there: one more rounding where the id occurs, nothing elsewhere
    base = torch.randn(V, H, generator=g).to(DEV)
    acc = B.embed_backward(plan, di, dY, dW=base.clone(), accumulate=True)
    off = np.abs(dev_to_f64(acc) - (dev_to_f64(base) + ref))
    assert np.all(off <= (64 + n / 16 + 16) * U * size + 2 * U * (np.abs(dev_to_f64(base)) + np.abs(ref)))
    gone = torch.from_numpy(n[:, 0] == 0).to(DEV)
    assert torch.equal(acc[gone], base[gone])
    return plan, W, di, dY, Y, dW


SIZES = [(1, 1, 1), (1, 1000, 64), (31, 2, 7), (32, 100, 100), (33, 3, 2048), (64, 64, 8), (2048, 100, 64),
         (2049, 1000, 24), (5000, 70000, 12), (4097, 1023, 136), (300, 1024, 300), (70, 50, 7168), (9000, 5, 40)]


@pytest.mark.parametrize("dtype", sorted(TYPES))
@pytest.mark.parametrize("kind", ["spread", "skewed"])
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
def test_against_oracle(size, kind, dtype):
    require_lib()
    check(*size, dtype, kind, seed=sum(size))


@pytest.mark.parametrize("kind", ["one", "down", "padded"])
@pytest.mark.parametrize("N", [5, 32, 64, 5000])
def test_one_id_all_ids_none(N, kind):
    require_lib()
    check(N, 777, 72, "bf16", kind)
    check(N, 777, 5, "f32", kind, scale=-0.5)


def test_many_positions_of_one_id():
    require_lib()
    check(70_000, 300, 16, "bf16", "skewed")
    check(70_000, 300, 8, "f32", "one")


def test_large_vocabularies_sort_in_more_passes():
    require_lib()
    check(3000, 2_000_000, 4, "f32", "spread")
    check(3000, 1 << 20, 8, "bf16", "skewed")


@pytest.mark.parametrize("dtype", sorted(TYPES))
def test_alignment_streams_and_neighbours(dtype):
    require_lib()
    plan, W, ids, dY, Y, dW = check(100, 60, 64, dtype, "skewed", seed=5)

    def shifted(t):
        flat = torch.full((t.numel() + 64,), -7, dtype=t.dtype, device=DEV)
        flat[1:1 + t.numel()] = t.reshape(-1)
        return flat[1:1 + t.numel()].view(t.shape), flat

    Ws, dYs, ids_s = shifted(W)[0], shifted(dY)[0], shifted(ids)[0]
    Yo, flat_Y = shifted(torch.zeros_like(Y))
    dWo, flat_W = shifted(torch.zeros_like(dW))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    B.embed_forward(plan, Ws, ids_s, Y=Yo, stream=s)
    B.embed_backward(plan, ids_s, dYs, dW=dWo, stream=s)
    s.synchronize()
    assert torch.equal(Yo, Y) and torch.equal(dWo, dW)
    for flat, t in ((flat_Y, Y), (flat_W, dW)):
        assert flat[0] == -7 and bool((flat[1 + t.numel():] == -7).all())


def test_rows_past_32_bit_offsets():
    """A table of more than 2^31 values: its last rows are found and written."""
    require_lib()
    V, H, N = 300_000, 7680, 40
    W = torch.zeros((V, H), dtype=torch.bfloat16, device=DEV)
    rows = torch.tensor([V - 1, V - 2, 279_621, 139_811, 0], device=DEV)
    W[rows] = torch.randn(5, H, device=DEV).bfloat16()
    ids = rows.repeat(8).int()
    plan = B.embed_plan(N, V, H, B.MOE_BF16, 1.0)
    assert torch.equal(B.embed_forward(plan, W, ids), W[ids.long()])
    dY = torch.randn(N, H, device=DEV).bfloat16()
    dW = B.embed_backward(plan, ids, dY)
    for i, v in enumerate(rows.tolist()):
        ref = dY[i::5].double().sum(0)
        assert torch.all((dW[v].double() - ref).abs() <= 80 * U * dY[i::5].double().abs().sum(0))
    dW[rows] = 0
    assert not dW.any()


def test_no_positions():
    require_lib()
    plan = B.embed_plan(0, 10, 64, B.MOE_F32)
    e, i = torch.empty((0, 64), device=DEV), torch.empty(0, dtype=torch.int32, device=DEV)
    assert not B.embed_backward(plan, i, e, dW=torch.ones((10, 64), device=DEV)).any()
    assert B.embed_backward(plan, i, e, dW=torch.ones((10, 64), device=DEV), accumulate=True).all()


def test_graph_replays():
    require_lib()
    from test_gpu_graph import capture, replay_and_check
    plan, W, ids, dY, Y, dW = check(3000, 500, 64, "bf16", "skewed")
    outs = {"Y": torch.empty_like(Y), "dW": torch.empty_like(dW)}
    ws = B.workspace(plan, "bwd", DEV)

    def call():
        B.embed_forward(plan, W, ids, outs["Y"])
        B.embed_backward(plan, ids, dY, outs["dW"], ws=ws)

    replay_and_check("embed", capture(call), outs, {"Y": Y, "dW": dW})


# Gradients larger than what is zeroed beside the sort (128 MB with up to 4096
# positions, 32 MB a launch with more), so that the summing launch zeroes the
# rest around the rows it writes: narrow and odd rows, pieces of 4096 rows.
PAST = [(3000, 1_200_000, 37, "bf16"), (5000, 700_000, 101, "f32"), (5000, 700_000, 101, "bf16"),
        (2000, 16_000_000, 3, "f32"), (4096, 140_000, 513, "bf16"), (20_000, 900_000, 72, "bf16")]


@pytest.mark.parametrize("size", PAST, ids=lambda s: "x".join(map(str, s)))
def test_rows_zeroed_around_those_that_occur(size):
    require_lib()
    N, V, H, dtype = size
    dt = TYPES[dtype]
    r = np.random.default_rng(V)
    ids = r.integers(0, V, N)
    ids[: N // 4] = V - 1 - r.integers(0, 300, N // 4)   # many near the end, some of them often
    ids[N // 4: N // 2] = V // 2 + np.arange(N // 2 - N // 4) % 977
    ids[-1], ids[-2], ids[-3] = V - 1, 0, -1
    di = torch.from_numpy(ids.astype(np.int32)).to(DEV)
    dY = torch.randn(N, H, generator=torch.Generator().manual_seed(N)).to(dt).to(DEV)
    plan = B.embed_plan(N, V, H, B.moe_dtype(dt), 0.5)
    dW = torch.full((V, H), float("nan"), device=DEV)
    B.embed_backward(plan, di, dY, dW=dW)
    ok = di >= 0
    rows, at, n = torch.unique(di[ok].long(), return_inverse=True, return_counts=True)
    dy = 0.5 * dY[ok].double()
    ref = torch.zeros((len(rows), H), dtype=torch.float64, device=DEV).index_add_(0, at, dy)
    size = torch.zeros_like(ref).index_add_(0, at, dy.abs())
    assert torch.all((dW[rows].double() - ref).abs() <= (64 + n[:, None] / 16 + 16) * U * size)
    sums = dW[rows]
    dW[rows] = 0
    assert not dW.any()  # NaN counts as something
    # onto ones: one rounding of the sum
    acc = torch.ones((V, H), device=DEV)
    B.embed_backward(plan, di, dY, dW=acc, accumulate=True)
    assert torch.all((acc[rows].double() - 1 - ref).abs() <= (64 + n[:, None] / 16 + 16) * U * size + 2 * U * (1 + ref.abs()))
    acc[rows] = 1
    assert bool((acc == 1).all()) and bool(torch.isfinite(sums).all())
