"""The operators around the layer on the host, without a GPU: exports, struct
layouts, plans, and argument errors before anything is enqueued."""

import ctypes
import os
import re
import subprocess
import tempfile

import pytest
import torch

from memory_bounded_expert_amd import binding as B

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

pytestmark = pytest.mark.skipif(not os.path.exists(B.LIB_PATH),
                                reason="libmoebound.so not built (run __graft_entry__.build())")

FAKE = ctypes.c_void_p(0x100000)  # never dereferenced: every check below fails first
PLANS = {"route_plan_t": B.RoutePlan, "lnorm_plan_t": B.LnormPlan, "embed_plan_t": B.EmbedPlan,
         "kd_plan_t": B.KdPlan}


def test_exports_and_argument_counts():
    L = B.lib()
    names = B.declared_operators()
    assert set(names) == {p + s for p in ("route_", "lnorm_", "embed_", "kd_")
                          for s in ("plan", "forward", "backward")} | {"moe_routed_forward",
                                                                       "moe_routed_backward"}
    for h in B.OPERATOR_HEADERS:
        text = re.sub(r"/\*.*?\*/", "", open(h).read(), flags=re.S)
        for m in re.finditer(r"\bint ([a-z]+_[a-z_]+)\s*\(([^;{]*?)\)\s*;", text, flags=re.S):
            name, params = m.group(1), m.group(2).strip()
            assert name in names
            assert len(getattr(L, name).argtypes) == params.count(",") + 1, name


@pytest.mark.parametrize("struct", sorted(PLANS))
def test_struct_layout_matches_c(struct):
    cls = PLANS[struct]
    src = ["#include <stdio.h>", "#include <stddef.h>"]
    src += ['#include "%s"' % os.path.basename(h) for h in B.OPERATOR_HEADERS]
    src += ["int main(void) {", 'printf("size %%zu\\n", sizeof(%s));' % struct]
    src += ['printf("%s %%zu\\n", offsetof(%s, %s));' % (n, struct, n) for n, _ in cls._fields_]
    src += ["return 0; }"]
    with tempfile.TemporaryDirectory() as d:
        c, exe = os.path.join(d, "t.c"), os.path.join(d, "t")
        open(c, "w").write("\n".join(src) + "\n")
        subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"),
                        c, "-o", exe], check=True)
        got = dict(l.split() for l in subprocess.run([exe], capture_output=True, text=True,
                                                     check=True).stdout.splitlines())
    assert int(got.pop("size")) == ctypes.sizeof(cls)
    for n, off in got.items():
        assert int(off) == getattr(cls, n).offset, n


# ---- routing

ROUTE_OK = dict(N=10, E=64, k=8, score=0, n_group=8, topk_group=4, group_top=2, renorm=1, scale=1.0)


@pytest.mark.parametrize("change,status", [
    (dict(N=-1), B.MOE_EINVAL), (dict(E=0, n_group=1), B.MOE_EINVAL), (dict(k=0), B.MOE_EINVAL),
    (dict(k=65), B.MOE_EINVAL), (dict(score=2), B.MOE_EINVAL), (dict(n_group=0), B.MOE_EINVAL),
    (dict(n_group=7), B.MOE_EINVAL), (dict(topk_group=0), B.MOE_EINVAL),
    (dict(topk_group=9), B.MOE_EINVAL), (dict(k=9, topk_group=1), B.MOE_EINVAL),
    (dict(group_top=0), B.MOE_EINVAL), (dict(group_top=3), B.MOE_EINVAL),
    (dict(renorm=2), B.MOE_EINVAL), (dict(scale=0.0), B.MOE_EINVAL),
    (dict(scale=-1.0), B.MOE_EINVAL), (dict(scale=float("inf")), B.MOE_EINVAL),
    (dict(scale=float("nan")), B.MOE_EINVAL),
    (dict(E=1032, n_group=1, topk_group=1), B.MOE_EUNSUPPORTED),
    (dict(E=128, k=65, n_group=1, topk_group=1), B.MOE_EUNSUPPORTED),
    (dict(E=130, k=2, n_group=65, topk_group=1), B.MOE_EUNSUPPORTED),
    (dict(N=2**26), B.MOE_EUNSUPPORTED),
])
def test_route_plan_errors(change, status):
    a = {**ROUTE_OK, **change}
    assert B.lib().route_plan(*a.values(), ctypes.byref(B.RoutePlan())) == status


def test_route_argument_errors():
    L, ref = B.lib(), ctypes.byref
    assert L.route_plan(*ROUTE_OK.values(), None) == B.MOE_EINVAL
    with pytest.raises(ValueError):
        B.route_plan(4, 8, 2, score="cosine")
    bad, p = B.RoutePlan(), B.route_plan(4, 8, 2)
    assert L.route_forward(ref(bad), FAKE, None, FAKE, FAKE, None) == B.MOE_EINVAL
    assert L.route_backward(ref(bad), FAKE, FAKE, FAKE, FAKE, None) == B.MOE_EINVAL
    for i in (0, 2, 3):
        args = [FAKE, None, FAKE, FAKE]
        args[i] = None
        assert L.route_forward(ref(p), *args, None) == B.MOE_EINVAL
    for i in range(4):
        args = [FAKE] * 4
        args[i] = None
        assert L.route_backward(ref(p), *args, None) == B.MOE_EINVAL
    p0 = B.route_plan(0, 8, 2)
    assert L.route_forward(ref(p0), *[None] * 5) == B.MOE_OK
    assert L.route_backward(ref(p0), *[None] * 5) == B.MOE_OK


def test_routed_layer_argument_errors():
    L, ref = B.lib(), ctypes.byref
    p = B.moe_plan_chunks(256, 64, 128, 8, 2, 64, 8, B.MOE_F32)
    fwd, bwd = [FAKE] * 7, [FAKE] * 12
    assert L.moe_routed_forward(ref(B.MoePlan()), *fwd, FAKE, 1 << 30, None, None) == B.MOE_EINVAL
    for i in range(7):
        args = list(fwd)
        args[i] = None
        assert L.moe_routed_forward(ref(p), *args, FAKE, 1 << 30, None, None) == B.MOE_EINVAL
    for i in range(12):
        args = list(bwd)
        args[i] = None
        assert L.moe_routed_backward(ref(p), *args, FAKE, 1 << 30, None, None) == B.MOE_EINVAL
    off = ctypes.c_void_p(0x100010)
    assert L.moe_routed_forward(ref(p), *fwd, off, 1 << 30, None, None) == B.MOE_EINVAL
    assert L.moe_routed_backward(ref(p), *bwd, off, 1 << 30, None, None) == B.MOE_EINVAL
    assert L.moe_routed_forward(ref(p), *fwd, FAKE, p.fwd_workspace_bytes - 1, None, None) == B.MOE_EWORKSPACE
    assert L.moe_routed_backward(ref(p), *bwd, FAKE, p.bwd_workspace_bytes - 1, None, None) == B.MOE_EWORKSPACE
    p0 = B.moe_plan_chunks(0, 64, 64, 8, 2, 4, 4, B.MOE_F32)
    st = B.MoeStats()
    assert L.moe_routed_forward(ref(p0), *[None] * 8, 0, None, ref(st)) == B.MOE_OK
    assert st.launches == 0


def test_routed_layer_refuses_matrices_off_a_16_byte_step():
    L, ref = B.lib(), ctypes.byref
    for dtype, by in ((B.MOE_F32, 4), (B.MOE_BF16, 2), (B.MOE_BF16, 8)):
        p = B.moe_plan_chunks(256, 64, 128, 8, 2, 64, 8, dtype)
        off = ctypes.c_void_p(0x100000 + by)
        for i in (0, 1, 2, 3, 6):
            args = [FAKE] * 7
            args[i] = off
            assert L.moe_routed_forward(ref(p), *args, FAKE, 1 << 30, None, None) == B.MOE_EINVAL
        for i in (0, 1, 2, 3, 4, 7, 8, 9, 10):
            args = [FAKE] * 12
            args[i] = off
            assert L.moe_routed_backward(ref(p), *args, FAKE, 1 << 30, None, None) == B.MOE_EINVAL


def test_binding_refuses_wrong_tensors():
    p = B.route_plan(4, 8, 2)
    l = torch.zeros(4, 8)
    for bad in (l[:3], l.double(), l.t().contiguous().t(), torch.zeros(8, 8)[::2]):
        with pytest.raises(ValueError):
            B.route_forward(p, bad)
    with pytest.raises(ValueError):  # not on a GPU
        B.route_forward(p, l)
    with pytest.raises(ValueError):
        B.route_forward(p, l, torch.zeros(7))
    with pytest.raises(ValueError):
        B.route_backward(p, l, torch.zeros(4, 2, dtype=torch.int64), torch.zeros(4, 2))


# ---- layer norm


@pytest.mark.parametrize("args,status", [
    ((-1, 64, 0, 1e-5), B.MOE_EINVAL), ((4, 0, 0, 1e-5), B.MOE_EINVAL), ((4, 64, 2, 1e-5), B.MOE_EINVAL),
    ((4, 64, 0, 0.0), B.MOE_EINVAL), ((4, 64, 0, float("nan")), B.MOE_EINVAL),
    ((4, 64, 0, float("inf")), B.MOE_EINVAL), ((4, 65537, 0, 1e-5), B.MOE_EUNSUPPORTED),
    ((2**31, 64, 0, 1e-5), B.MOE_EUNSUPPORTED),
])
def test_lnorm_plan_errors(args, status):
    assert B.lib().lnorm_plan(*args, ctypes.byref(B.LnormPlan())) == status


def test_lnorm_argument_errors():
    L, ref = B.lib(), ctypes.byref
    assert L.lnorm_plan(4, 64, 0, 1e-5, None) == B.MOE_EINVAL
    p, big = B.lnorm_plan(4, 64, B.MOE_F32), 1 << 30
    assert L.lnorm_forward(ref(B.LnormPlan()), *[FAKE] * 6, None) == B.MOE_EINVAL
    assert L.lnorm_backward(ref(B.LnormPlan()), *[FAKE] * 9, big, None) == B.MOE_EINVAL
    for i in (0, 1, 3, 4, 5):
        args = [FAKE] * 6
        args[i] = None
        assert L.lnorm_forward(ref(p), *args, None) == B.MOE_EINVAL
    for i in (0, 1, 2, 3, 4, 5, 6, 8):
        args = [FAKE] * 9
        args[i] = None
        assert L.lnorm_backward(ref(p), *args, big, None) == B.MOE_EINVAL
    assert L.lnorm_backward(ref(p), *[FAKE] * 8, ctypes.c_void_p(0x100080), big, None) == B.MOE_EINVAL
    assert L.lnorm_backward(ref(p), *[FAKE] * 9, p.bwd_workspace_bytes - 1, None) == B.MOE_EWORKSPACE
    p0 = B.lnorm_plan(0, 64, B.MOE_F32)
    assert L.lnorm_forward(ref(p0), *[None] * 7) == B.MOE_OK
    assert L.lnorm_backward(ref(p0), *[None] * 9, 0, None) == B.MOE_EINVAL  # dgamma


def test_lnorm_binding_refuses_wrong_tensors():
    p = B.lnorm_plan(4, 64, B.MOE_F32)
    x, g = torch.zeros(4, 64), torch.zeros(64)
    for bad in (x[:3], x.bfloat16(), torch.zeros(4, 128)[:, ::2], torch.zeros(64, 4).t()):
        with pytest.raises(ValueError):
            B.lnorm_forward(p, bad, g)
    with pytest.raises(ValueError):
        B.lnorm_forward(p, x, g.bfloat16())
    with pytest.raises(ValueError):  # not on a GPU
        B.lnorm_forward(p, x, g)


# ---- token embedding


@pytest.mark.parametrize("args,status", [
    ((-1, 10, 64, 0, 1.0), B.MOE_EINVAL), ((4, 0, 64, 0, 1.0), B.MOE_EINVAL),
    ((4, 10, 0, 0, 1.0), B.MOE_EINVAL), ((4, 10, 64, 3, 1.0), B.MOE_EINVAL),
    ((4, 10, 64, 0, float("nan")), B.MOE_EINVAL), ((4, 10, 64, 0, float("inf")), B.MOE_EINVAL),
    ((2**26, 10, 64, 0, 1.0), B.MOE_EUNSUPPORTED), ((4, 2**30, 64, 0, 1.0), B.MOE_EUNSUPPORTED),
    ((4, 10, 65537, 0, 1.0), B.MOE_EUNSUPPORTED),
])
def test_embed_plan_errors(args, status):
    assert B.lib().embed_plan(*args, ctypes.byref(B.EmbedPlan())) == status


def test_embed_argument_errors():
    L, ref = B.lib(), ctypes.byref
    assert L.embed_plan(4, 10, 64, 0, 1.0, None) == B.MOE_EINVAL
    p, big = B.embed_plan(4, 10, 64, B.MOE_F32), 1 << 30
    assert L.embed_forward(ref(B.EmbedPlan()), *[FAKE] * 3, None) == B.MOE_EINVAL
    assert L.embed_backward(ref(B.EmbedPlan()), *[FAKE] * 3, 0, FAKE, big, None) == B.MOE_EINVAL
    for i in range(3):
        args = [FAKE] * 3
        args[i] = None
        assert L.embed_forward(ref(p), *args, None) == B.MOE_EINVAL
        assert L.embed_backward(ref(p), *args, 0, FAKE, big, None) == B.MOE_EINVAL
    assert L.embed_backward(ref(p), *[FAKE] * 3, 0, None, big, None) == B.MOE_EINVAL
    assert L.embed_backward(ref(p), *[FAKE] * 3, 0, ctypes.c_void_p(0x100004), big, None) == B.MOE_EINVAL
    assert L.embed_backward(ref(p), *[FAKE] * 3, 0, FAKE, p.bwd_workspace_bytes - 1, None) == B.MOE_EWORKSPACE
    p0 = B.embed_plan(0, 10, 64, B.MOE_F32)
    assert L.embed_forward(ref(p0), *[None] * 4) == B.MOE_OK
    assert L.embed_backward(ref(p0), *[None] * 3, 0, None, 0, None) == B.MOE_EINVAL  # dW
    assert L.embed_backward(ref(p0), None, None, FAKE, 1, None, 0, None) == B.MOE_OK


def test_embed_binding_refuses_wrong_tensors():
    p = B.embed_plan(4, 10, 64, B.MOE_F32)
    W, ids = torch.zeros(10, 64), torch.zeros(4, dtype=torch.int32)
    for w, i in ((W[:9], ids), (W.bfloat16(), ids), (W, ids.long()), (W, ids[:3]), (W, ids)):
        with pytest.raises(ValueError):  # the last pair is not on a GPU
            B.embed_forward(p, w, i)
    with pytest.raises(ValueError):
        B.embed_backward(p, ids, torch.zeros(4, 64), accumulate=True)


# ---- distillation

KD_OK = dict(N=8, H=128, V=1000, v_chunk=256, K=16, temperature=1.0, dtype=1, dw_dtype=0)


@pytest.mark.parametrize("change,status", [
    (dict(N=-1), B.MOE_EINVAL), (dict(H=0), B.MOE_EINVAL), (dict(V=0), B.MOE_EINVAL),
    (dict(v_chunk=0), B.MOE_EINVAL), (dict(K=0), B.MOE_EINVAL), (dict(temperature=0.0), B.MOE_EINVAL),
    (dict(temperature=-2.0), B.MOE_EINVAL), (dict(temperature=float("nan")), B.MOE_EINVAL),
    (dict(temperature=float("inf")), B.MOE_EINVAL), (dict(dtype=2), B.MOE_EINVAL),
    (dict(dw_dtype=5), B.MOE_EINVAL), (dict(dtype=0), B.MOE_EUNSUPPORTED),
    (dict(H=192), B.MOE_EUNSUPPORTED), (dict(v_chunk=300), B.MOE_EUNSUPPORTED),
    (dict(K=257), B.MOE_EUNSUPPORTED), (dict(N=2**23), B.MOE_EUNSUPPORTED),
    (dict(v_chunk=2**23), B.MOE_EUNSUPPORTED), (dict(V=2**31), B.MOE_EUNSUPPORTED),
    (dict(N=2**16, v_chunk=2**14), B.MOE_EUNSUPPORTED),
])
def test_kd_plan_errors(change, status):
    assert B.lib().kd_plan(*{**KD_OK, **change}.values(), ctypes.byref(B.KdPlan())) == status


def test_kd_workspaces_hold_the_strip_and_the_sums_alone():
    pad = lambda n: -(-n // 256) * 256
    for N, H, V, v_chunk in ((8192, 7168, 200_000, 8192), (8200, 640, 10_001, 1024), (777, 512, 20_000, 4096),
                             (1, 128, 10, 256), (16, 4096, 100_000, 1024), (2000, 1024, 150_000, 256)):
        p = B.kd_plan(N, H, V, v_chunk, 32)
        strip = pad(N * min(p.strip, -(-V // 256) * 256) * 2)
        tiles = -(-N // 256) * (H // (256 if H % 256 == 0 else 128))
        sums = p.bwd_workspace_bytes - strip  # whole sums of dX; one, or what fills the chip once
        if tiles > 128:
            assert sums == pad(4 * N * H)
        else:
            assert pad(4 * N * H) <= sums <= pad(4 * N * H * (256 // tiles)) <= 64 << 20
    # the forward pass: two statistics for each 128 columns of its strip, and two a token
    p, q = (B.kd_plan(8192, 7168, 200_000, c, 32) for c in (8192, 16_384))
    assert p.fwd_workspace_bytes == q.fwd_workspace_bytes == 2 * (8192 // 128) * 8192 * 4 + 2 * 8192 * 4


def test_kd_temperatures_without_a_reciprocal():
    for T, status in ((1e-39, B.MOE_EINVAL), (1e-38, B.MOE_OK), (3e38, B.MOE_OK)):
        assert B.lib().kd_plan(*{**KD_OK, "temperature": T}.values(), ctypes.byref(B.KdPlan())) == status


def test_kd_strips_and_workspace():
    p = B.kd_plan(8192, 7168, 200_000, 8192, 32)
    c = B.cce_plan(8192, 7168, 200_000, 8192)
    assert (p.S, p.strip_bound_bytes) == (c.S, c.strip_bound_bytes) == (25, 8192 * 8192 * 2)
    # beside the cross-entropy's: the list's probabilities
    assert p.bwd_workspace_bytes <= c.bwd_workspace_bytes + 8192 * 32 * 4 + 256
    assert p.fwd_workspace_bytes <= c.fwd_workspace_bytes
    # a small batch takes wider strips, within the bound
    for N, H, V, v_chunk in ((777, 512, 20_000, 4096), (16, 7168, 200_000, 1024), (2000, 1024, 150_000, 256), (1, 128, 10, 256)):
        p = B.kd_plan(N, H, V, v_chunk, 4)
        assert p.strip % v_chunk == 0 and p.S == -(-V // p.strip)
        assert p.strip == v_chunk or p.strip_bound_bytes <= 64 << 20
        most = min((64 << 20) // (2 * N), ((1 << 30) - 1) // H)  # columns that fit
        assert p.S <= -(-V // max(most // v_chunk * v_chunk, v_chunk)) or p.S == 1


def test_kd_argument_errors():
    L, ref = B.lib(), ctypes.byref
    assert L.kd_plan(*KD_OK.values(), None) == B.MOE_EINVAL
    p, big = B.kd_plan(**KD_OK), 1 << 30
    assert L.kd_forward(ref(B.KdPlan()), *[FAKE] * 8, big, None) == B.MOE_EINVAL
    assert L.kd_backward(ref(B.KdPlan()), *[FAKE] * 10, big, None) == B.MOE_EINVAL
    for n, f in ((8, L.kd_forward), (10, L.kd_backward)):
        for i in range(n):
            args = [FAKE] * n
            args[i] = None
            assert f(ref(p), *args, big, None) == B.MOE_EINVAL
        assert f(ref(p), *[FAKE] * (n - 1), ctypes.c_void_p(0x100080), big, None) == B.MOE_EINVAL
    off = ctypes.c_void_p(0x100008)
    for i in (0, 1):
        args = [FAKE] * 8
        args[i] = off
        assert L.kd_forward(ref(p), *args, big, None) == B.MOE_EINVAL
    for i in (0, 1, 7, 8):
        args = [FAKE] * 10
        args[i] = off
        assert L.kd_backward(ref(p), *args, big, None) == B.MOE_EINVAL
    assert L.kd_forward(ref(p), *[FAKE] * 8, p.fwd_workspace_bytes - 1, None) == B.MOE_EWORKSPACE
    assert L.kd_backward(ref(p), *[FAKE] * 10, p.bwd_workspace_bytes - 1, None) == B.MOE_EWORKSPACE
    p0 = B.kd_plan(**{**KD_OK, "N": 0})
    assert L.kd_forward(ref(p0), *[None] * 8, 0, None) == B.MOE_OK
    assert L.kd_backward(ref(p0), *[None] * 10, 0, None) == B.MOE_EINVAL  # dW


def test_kd_binding_refuses_wrong_tensors():
    p = B.kd_plan(**KD_OK)
    ok = dict(X=torch.zeros(8, 128).bfloat16(), W=torch.zeros(1000, 128).bfloat16(),
              t_idx=torch.zeros(8, 16, dtype=torch.int32), t_logit=torch.zeros(8, 16))
    for change in (dict(X=torch.zeros(8, 128)), dict(W=ok["W"][:999]), dict(t_idx=ok["t_idx"].long()),
                   dict(t_logit=ok["t_logit"][:, :8]), dict()):  # the last: not on a GPU
        with pytest.raises(ValueError):
            B.kd_forward(p, **{**ok, **change})


def test_binding_refuses_a_workspace_elsewhere():
    with pytest.raises(ValueError):
        B._workspace(torch.empty(1 << 20, dtype=torch.uint8), B.lnorm_plan(4, 64, B.MOE_F32), "bwd", torch.device("cuda:0"))
    with pytest.raises(ValueError):
        B._workspace(torch.empty((64, 64), dtype=torch.uint8)[:, ::2], B.lnorm_plan(4, 64, B.MOE_F32), "bwd", torch.device("cpu"))
