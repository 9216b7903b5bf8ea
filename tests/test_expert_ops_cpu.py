"""The 8-bit path of an expert layer on the host, without a GPU: exports, struct layouts, plans, and argument errors
before anything is enqueued."""

import ctypes
import os
import re
import shutil
import subprocess

import pytest
import torch

from memory_bounded_expert_amd import binding as B
from test_plans_host import CSRC, HIPCC, INCLUDE, ROOT, STUBS, SWEEP

pytestmark = pytest.mark.skipif(not os.path.exists(B.LIB_PATH), reason="libmoebound.so not built (run __graft_entry__.build())")

FAKE = ctypes.c_void_p(0x100000)  # never dereferenced: every check below fails first
PLANS = {"rms_plan_t": B.RmsPlan, "q8_plan_t": B.Q8Plan, "gmm_plan_t": B.GmmPlan}
ref = ctypes.byref


def test_exports_and_argument_counts():
    L, names = B.lib(), B.declared_expert_operators()
    assert set(names) == {"rms_plan", "rms_forward", "rms_forward_q8", "rms_backward", "q8_plan", "q8_pack", "q8_unpack",
                          "q8_pack_weights", "q8_swiglu_forward", "q8_swiglu_backward", "gmm_plan", "gmm_forward",
                          "gmm_backward_dx", "gmm_backward_dw", "gmm8_forward", "gmm8_backward_dw"}
    seen = set()
    for h in B.EXPERT_HEADERS:
        text = re.sub(r"/\*.*?\*/", "", open(h).read(), flags=re.S)
        for name, params in re.findall(r"\bint ([a-z0-9]+_[a-z0-9_]+)\s*\(([^;{]*?)\)\s*;", text, flags=re.S):
            assert len(getattr(L, name).argtypes) == params.count(",") + 1, name
            seen.add(name)
    assert seen == set(names)


@pytest.mark.parametrize("struct", sorted(PLANS))
def test_struct_layout_matches_c(struct, tmp_path):
    cls = PLANS[struct]
    src = ["#include <stdio.h>", "#include <stddef.h>"] + ['#include "%s"' % os.path.basename(h) for h in B.EXPERT_HEADERS]
    src += ["int main(void) {", 'printf("size %%zu\\n", sizeof(%s));' % struct]
    src += ['printf("%s %%zu\\n", offsetof(%s, %s));' % (n, struct, n) for n, _ in cls._fields_] + ["return 0; }"]
    c, exe = str(tmp_path / "t.c"), str(tmp_path / "t")
    open(c, "w").write("\n".join(src) + "\n")
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), c, "-o", exe], check=True)
    got = dict(l.split() for l in subprocess.run([exe], capture_output=True, text=True, check=True).stdout.splitlines())
    assert int(got.pop("size")) == ctypes.sizeof(cls)
    for n, off in got.items():
        assert int(off) == getattr(cls, n).offset, n


def test_what_the_8_bit_product_cuts_is_stated(tmp_path):
    """The header's bound of gmm8_forward's sums is the binding's: 2^-13 for each of seven products of eight."""
    c, exe = str(tmp_path / "t.c"), str(tmp_path / "t")
    open(c, "w").write('#include <stdio.h>\n#include "gmm.h"\nint main(void) { printf("%.17g\\n", GMM8_CUT); return 0; }\n')
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), c, "-o", exe], check=True)
    out = subprocess.run([exe], capture_output=True, text=True, check=True).stdout
    assert float(out) == B.GMM8_CUT == 7 * 2.0 ** -13


CALLS = {
    "rms": ("rms", "rms.h", "ROWS(N) SIZES(H) for (int d = -1; d < 3; ++d) { rms_plan_t p; ok += rms_plan(N, H, d, 1e-5f, &p) == MOE_OK; }"),
    "q8": ("q8", "q8.h", "ROWS(N) SIZES(H) for (int d = -1; d < 3; ++d) { q8_plan_t p; ok += q8_plan(N, H, d, &p) == MOE_OK; }"),
    "gmm": ("gmm", "gmm.h", "ROWS(R) SIZES(K) SIZES(N) SIZES(E) for (int d = -1; d < 3; ++d) { gmm_plan_t p; ok += gmm_plan(R, K, N, E, d, &p) == MOE_OK; }"),
}


@pytest.mark.skipif(not os.path.exists(HIPCC) or not shutil.which("gcc"), reason="no hipcc")
@pytest.mark.parametrize("name", sorted(CALLS))
def test_plans_do_nothing_undefined(name, tmp_path):
    """As test_plans_host.py: undefined arithmetic traps, from no rows to past the limits."""
    source, header, calls = CALLS[name]
    obj, main, exe = (str(tmp_path / n) for n in ("plan.o", "main.c", "main"))
    subprocess.run([HIPCC, "--offload-host-only", "-O1", "-std=c++17", "-fPIC", f"-I{INCLUDE}", f"-I{CSRC}",
                    "-Xarch_host", "-fsanitize=undefined", "-Xarch_host", "-fsanitize-trap=undefined",
                    "-c", os.path.join(CSRC, source + ".hip"), "-o", obj], check=True)
    open(main, "w").write('#include "%s"\n' % header + STUBS + SWEEP.replace("CALLS", calls))
    subprocess.run(["gcc", "-std=c99", f"-I{INCLUDE}", main, obj, "-o", exe, "-lstdc++", "-lm", "-Wl,--unresolved-symbols=ignore-all"], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, f"{name}: a plan's arithmetic trapped ({r.returncode})"
    assert int(r.stdout) > 20


# ---- plans


@pytest.mark.parametrize("a,status", [
    ((-1, 8, 1, 1e-6), B.MOE_EINVAL), ((1, 0, 1, 1e-6), B.MOE_EINVAL), ((1, 8, 2, 1e-6), B.MOE_EINVAL), ((1, 8, 1, 0.0), B.MOE_EINVAL),
    ((1, 8, 1, -1.0), B.MOE_EINVAL), ((1, 8, 1, float("inf")), B.MOE_EINVAL), ((1, 8, 1, float("nan")), B.MOE_EINVAL),
    ((1, 65537, 1, 1e-6), B.MOE_EUNSUPPORTED), ((2 ** 31, 8, 1, 1e-6), B.MOE_EUNSUPPORTED), ((0, 1, 0, 1e-6), B.MOE_OK)])
def test_rms_plan_errors(a, status):
    assert B.lib().rms_plan(*a, ref(B.RmsPlan())) == status
    assert B.lib().rms_plan(*a, None) == B.MOE_EINVAL


@pytest.mark.parametrize("a,status", [
    ((-1, 8, 1), B.MOE_EINVAL), ((1, 0, 1), B.MOE_EINVAL), ((1, 8, 2), B.MOE_EINVAL), ((1, 65537, 1), B.MOE_EUNSUPPORTED),
    ((2 ** 31, 8, 1), B.MOE_EUNSUPPORTED), ((0, 1, 0), B.MOE_OK)])
def test_q8_plan_errors(a, status):
    assert B.lib().q8_plan(*a, ref(B.Q8Plan())) == status
    assert B.lib().q8_plan(*a, None) == B.MOE_EINVAL


@pytest.mark.parametrize("h,row,scale", [(1, 128, 4), (127, 128, 4), (128, 128, 4), (129, 256, 4), (512, 512, 4), (513, 640, 8), (7168, 7168, 56)])
def test_q8_pitches(h, row, scale):
    for p in (B.q8_plan(3, h), B.rms_plan(3, h)):
        assert (p.row_pitch, p.scale_pitch) == (row, scale)
    assert B.gmm_plan(3, h, 8, 1, B.GMM_Q8).row_pitch == row


@pytest.mark.parametrize("a,status", [
    ((-1, 8, 8, 1, 0), B.MOE_EINVAL), ((1, 0, 8, 1, 0), B.MOE_EINVAL), ((1, 8, 0, 1, 0), B.MOE_EINVAL), ((1, 8, 8, -1, 0), B.MOE_EINVAL),
    ((1, 8, 8, 0, 0), B.MOE_EINVAL), ((1, 8, 8, 1, 2), B.MOE_EINVAL), ((1, 8, 8, 1, -1), B.MOE_EINVAL), ((1, 12, 8, 1, 0), B.MOE_EINVAL),
    ((1, 8, 12, 1, 0), B.MOE_EINVAL), ((1, 8, 12, 1, 1), B.MOE_EINVAL), ((1, 9, 8, 1, 1), B.MOE_OK), ((0, 8, 8, 0, 0), B.MOE_OK),
    ((1, 65544, 8, 1, 0), B.MOE_EUNSUPPORTED), ((1, 8, 65544, 1, 0), B.MOE_EUNSUPPORTED), ((1, 8, 8, 1025, 0), B.MOE_EUNSUPPORTED),
    ((2 ** 31 - 65536, 8, 8, 1, 0), B.MOE_EUNSUPPORTED), ((1, 65536, 65536, 1, 0), B.MOE_EUNSUPPORTED), ((1, 32768, 32768, 1, 1), B.MOE_EUNSUPPORTED),
    ((2 ** 30, 65536, 8, 1, 0), B.MOE_EUNSUPPORTED)])
def test_gmm_plan_errors(a, status):
    assert B.lib().gmm_plan(*a, ref(B.GmmPlan())) == status
    assert B.lib().gmm_plan(*a, None) == B.MOE_EINVAL


@pytest.mark.parametrize("operands", [B.GMM_BF16, B.GMM_Q8])
def test_gmm_plans_whose_launch_would_be_refused(operands):
    """256 rows of one column tile are 512 threads, and an expert's rows may end in a tile of their own: HIP takes fewer
    than 2^32 threads of a launch."""
    plan = lambda R, K, N, E: B.lib().gmm_plan(R, K, N, E, operands, ref(B.GmmPlan()))
    most = 2 ** 31 - 65536 - 1
    for E in (1, 64, 255):
        assert (most // 256 + E) * 512 < 2 ** 32 and plan(most, 8, 8, E) == B.MOE_OK
    for E in (257, 512, 1024):
        assert (most // 256 + E) * 512 >= 2 ** 32 and plan(most, 8, 8, E) == B.MOE_EUNSUPPORTED
    R = 2 ** 31 - 512 * 1024 // 2 - 256
    assert (R // 256 + 1024) * 512 < 2 ** 32 and plan(R, 8, 8, 1024) == B.MOE_OK
    assert plan(2 ** 31 - 512 * 1024 // 2, 8, 8, 1024) == B.MOE_EUNSUPPORTED
    for R in (0, 1, 300, 100_000):  # and of dW's, whatever the rows
        assert plan(R, 32768, 32760, 1024) == (B.MOE_EUNSUPPORTED if 16384 * 1024 * 512 >= 2 ** 32 else B.MOE_OK)
    # dX's columns are K
    if operands == B.GMM_BF16:
        assert plan(2 ** 30, 512, 8, 1024) == B.MOE_EUNSUPPORTED and plan(2 ** 30, 256, 8, 1024) == B.MOE_OK


# ---- calls


def refuses(f, plan, args, tail=(None,), status=B.MOE_EINVAL):
    assert f(ref(plan), *args, *tail) == status, (f.__name__, args)


def each_without(args, skip=()):
    for i in range(len(args)):
        if i not in skip:
            yield [None if j == i else a for j, a in enumerate(args)]


def off(by):
    return ctypes.c_void_p(0x100000 + by)


def test_rms_argument_errors():
    L, p = B.lib(), B.rms_plan(4, 8)
    for f, n, tail in ((L.rms_forward, 6, ()), (L.rms_forward_q8, 7, ()), (L.rms_backward, 8, (1 << 30,))):
        refuses(f, B.RmsPlan(), [FAKE] * n, (*tail, None))
    # X, residual, gamma, S, Y, rstd: a residual without S, S without a residual, and what is required
    for args in each_without([FAKE] * 6):
        refuses(L.rms_forward, p, args)
    for args in each_without([FAKE] * 7):
        refuses(L.rms_forward_q8, p, args)
    for i, by in ((4, 8), (5, 2)):
        args = [FAKE] * 7
        args[i] = off(by)
        refuses(L.rms_forward_q8, p, args)
    # S, gamma, dY, rstd, dS (may be NULL), dX, dgamma, workspace
    for args in each_without([FAKE] * 8, skip=(4,)):
        refuses(L.rms_backward, p, args, (1 << 30, None))
    refuses(L.rms_backward, p, [FAKE] * 7 + [off(16)], (1 << 30, None))
    refuses(L.rms_backward, p, [FAKE] * 8, (p.bwd_workspace_bytes - 1, None), B.MOE_EWORKSPACE)
    refuses(L.rms_backward, B.rms_plan(0, 8), [None] * 8, (0, None))
    p0 = B.rms_plan(0, 8)
    assert L.rms_forward(ref(p0), *[None] * 7) == B.MOE_OK and L.rms_forward_q8(ref(p0), *[None] * 8) == B.MOE_OK


def test_q8_argument_errors():
    L = B.lib()
    for dtype, size in ((B.MOE_BF16, 2), (B.MOE_F32, 4)):
        p, bad = B.q8_plan(4, 8, dtype), B.Q8Plan()
        # (call, arguments, which are q (16 bytes) and s (4 bytes), which have the element's alignment)
        for f, n, qs, ss, es in ((L.q8_pack, 3, (1,), (2,), (0,)), (L.q8_unpack, 3, (0,), (1,), (2,)),
                                 (L.q8_swiglu_forward, 8, (2, 4, 6), (3, 5, 7), (0, 1)), (L.q8_swiglu_backward, 7, (0, 2), (1, 3), (4, 5, 6))):
            refuses(f, bad, [FAKE] * n)
            for args in each_without([FAKE] * n):
                refuses(f, p, args)
            for places, by in ((qs, 8), (ss, 2), (es, size // 2)):
                for i in places:
                    args = [FAKE] * n
                    args[i] = off(by)
                    refuses(f, p, args)
            assert f(ref(B.q8_plan(0, 8, dtype)), *[None] * (n + 1)) == B.MOE_OK


def test_q8_weights_argument_errors():
    f = B.lib().q8_pack_weights
    call = lambda E=2, K=8, N=8, dtype=1, W=FAKE, q=FAKE, s=FAKE, qt=FAKE, st=FAKE: f(E, K, N, dtype, W, q, s, qt, st, None)
    for bad in (dict(E=-1), dict(K=0), dict(N=0), dict(dtype=2), dict(W=None), dict(q=None), dict(s=None), dict(qt=None), dict(st=None),
                dict(q=None, s=None, qt=None, st=None), dict(W=off(1)), dict(q=off(8)), dict(s=off(2)), dict(qt=off(8)), dict(st=off(2))):
        assert call(**bad) == B.MOE_EINVAL, bad
    for bad in (dict(K=65537), dict(N=65537), dict(E=65536)):
        assert call(**bad) == B.MOE_EUNSUPPORTED, bad
    assert call(E=0, W=None, q=None, s=None, qt=None, st=None) == B.MOE_OK


GMM = {  # matrices (16-byte aligned), scales, then offsets and the output come in this order
    "gmm_forward": (B.GMM_BF16, 2, ()), "gmm_backward_dx": (B.GMM_BF16, 2, ()), "gmm_backward_dw": (B.GMM_BF16, 2, ()),
    "gmm8_forward": (B.GMM_Q8, 4, (1, 3)), "gmm8_backward_dw": (B.GMM_Q8, 3, (1,))}


@pytest.mark.parametrize("name", sorted(GMM))
def test_gmm_argument_errors(name):
    operands, n, scales = GMM[name]
    f, p = getattr(B.lib(), name), B.gmm_plan(4, 16, 8, 3, operands)
    dw = name.endswith("dw")
    tail = ((0,) if dw else ()) + (FAKE, 1 << 40, None)
    args = [FAKE] * (n + 2)
    refuses(f, B.GmmPlan(), args, tail)
    refuses(f, B.gmm_plan(4, 16, 8, 3, 1 - operands), args, tail)
    for a in each_without(args):
        refuses(f, p, a, tail)
    for i in range(n + 2):
        by = 2 if i in scales or i == n else 8
        refuses(f, p, [off(by) if j == i else FAKE for j in range(n + 2)], tail)
    # nothing to do: no rows (dW is written all the same), no experts
    p0 = B.gmm_plan(0, 16, 8, 3, operands)
    if dw:
        refuses(f, p0, [None] * (n + 2), (0, None, 0, None))
    else:
        assert f(ref(p0), *[None] * (n + 3), 0, None) == B.MOE_OK
    none = B.gmm_plan(0, 16, 8, 0, operands)
    assert f(ref(none), *[None] * (n + 2), *((0,) if dw else ()), None, 0, None) == B.MOE_OK


@pytest.mark.parametrize("name", sorted(GMM))
def test_gmm_workspaces(name):
    """Wherever the plan asks for a workspace, a call refuses one that is missing, off its step or too small."""
    operands, n, _ = GMM[name]
    f, dw, asked = getattr(B.lib(), name), name.endswith("dw"), 0
    for R in (1, 8, 64, 300, 5000):
        for K in (64, 2048, 16384):
            for E in (1, 4):
                p = B.gmm_plan(R, K, 2048, E, operands)
                need = p.bwd_workspace_bytes if dw else p.fwd_workspace_bytes
                if not need:
                    continue
                asked += 1
                pre = (0,) if dw else ()
                refuses(f, p, [FAKE] * (n + 2), (*pre, None, need, None))
                refuses(f, p, [FAKE] * (n + 2), (*pre, off(128), need, None))
                refuses(f, p, [FAKE] * (n + 2), (*pre, FAKE, need - 1, None), B.MOE_EWORKSPACE)
    print(name, "plans with a workspace:", asked)


def test_binding_refuses_wrong_tensors():
    z = lambda *s, d=torch.bfloat16: torch.zeros(*s, dtype=d)
    q = lambda *s: z(*s, d=torch.uint8).view(B.E4M3)
    s8 = lambda *s: z(*s, d=torch.uint8).view(B.E8M0)
    rp, qp, gp, g8 = B.rms_plan(4, 16), B.q8_plan(4, 16), B.gmm_plan(4, 16, 8, 2), B.gmm_plan(4, 16, 8, 2, B.GMM_Q8)
    x, ga, of = z(4, 16), z(16, d=torch.float32), z(3, d=torch.int32)
    bad_calls = [
        lambda: B.rms_forward(rp, x[:3], ga), lambda: B.rms_forward(rp, x.float(), ga), lambda: B.rms_forward(rp, x, ga.bfloat16()),
        lambda: B.rms_forward(rp, x, ga, S=x), lambda: B.rms_forward(rp, x, ga, residual=x[:2]), lambda: B.rms_forward(rp, x, ga),
        lambda: B.rms_backward(rp, x, ga, x, z(4), x), lambda: B.rms_backward(rp, x, ga, x, z(4, d=torch.float32), dS=x.float()),
        lambda: B.q8_pack(qp, x.t().contiguous().t()), lambda: B.q8_pack(qp, x), lambda: B.q8_unpack(qp, q(4, 16), s8(4, 4)),
        lambda: B.q8_unpack(qp, q(4, 128), s8(4, 1)), lambda: B.q8_unpack(qp, z(4, 128, d=torch.uint8), s8(4, 4)),
        lambda: B.q8_pack_weights(z(2, 8, 8), "M"), lambda: B.q8_pack_weights(z(8, 8)), lambda: B.q8_pack_weights(z(2, 8, 8).half()),
        lambda: B.q8_swiglu_forward(qp, x, x[:3]), lambda: B.q8_swiglu_backward(qp, (q(4, 128), s8(4, 4), q(4, 128), s8(4, 3)), x),
        lambda: B.gmm_forward(gp, x, z(2, 16, 8)), lambda: B.gmm_forward(gp, x, z(2, 8, 16), of), lambda: B.gmm_forward(gp, x, z(2, 16, 8), of.long()),
        lambda: B.gmm_forward(gp, x, z(2, 16, 8), of[:2]), lambda: B.gmm_backward_dx(gp, x, z(2, 16, 8), of),
        lambda: B.gmm_backward_dw(gp, x, x, of), lambda: B.gmm_backward_dw(gp, x, z(4, 8), of, accumulate=True),
        lambda: B.gmm_forward(gp, x, z(2, 16, 8), of),  # not on a GPU
        lambda: B.gmm8_forward(g8, q(4, 128), s8(4, 4), q(2, 8, 128), s8(2, 2, 4), of), lambda: B.gmm8_forward(gp, q(4, 128), s8(4, 4), q(2, 8, 128), s8(2, 1, 4), of),
        lambda: B.gmm8_backward_dw(g8, q(4, 128), s8(4, 4), z(4, 16), of),
    ]
    for i, call in enumerate(bad_calls):
        with pytest.raises(ValueError):
            call()
            print("call", i, "passed")


def test_binding_says_what_is_wrong():
    """Each refusal by its own check: the name of the tensor and what does not fit, before the look at the device."""
    z = lambda *s, d=torch.bfloat16: torch.zeros(*s, dtype=d)
    q = lambda *s: z(*s, d=torch.uint8).view(B.E4M3)
    s8 = lambda *s: z(*s, d=torch.uint8).view(B.E8M0)
    f32 = torch.float32
    rp, qp, gp, g8 = B.rms_plan(4, 16), B.q8_plan(4, 16), B.gmm_plan(4, 16, 8, 2), B.gmm_plan(4, 16, 8, 2, B.GMM_Q8)
    x, dy, ga, w, of = z(4, 16), z(4, 8), z(16, d=f32), z(2, 16, 8), z(3, d=torch.int32)
    xq, xs, wq, ws = q(4, 128), s8(4, 4), q(2, 8, 128), s8(2, 1, 4)
    odd = z(16, 4).t()  # 4 x 16, not in one piece
    kept = (xq, xs, xq, xs)
    meta = lambda t: t.to("meta")
    for message, call in (
            ("^X: shape", lambda: B.rms_forward(rp, x[:3], ga)), ("^X: dtype", lambda: B.rms_forward(rp, x.float(), ga)),
            ("^X must be contiguous", lambda: B.rms_forward(rp, odd, ga)), ("^gamma: dtype", lambda: B.rms_forward(rp, x, ga.bfloat16())),
            ("^gamma: shape", lambda: B.rms_forward(rp, x, ga[:8])), ("^gamma: device", lambda: B.rms_forward(rp, x, meta(ga))),
            ("^residual: shape", lambda: B.rms_forward(rp, x, ga, residual=x[:2])), ("^residual: dtype", lambda: B.rms_forward_q8(rp, x, ga, x.float())),
            ("^S is X itself", lambda: B.rms_forward(rp, x, ga, S=x)), ("^S is X itself", lambda: B.rms_forward_q8(rp, x, ga, S=x)),
            ("^dY: shape", lambda: B.rms_backward(rp, x, ga, x[:1], ga[:4])), ("^rstd: dtype", lambda: B.rms_backward(rp, x, ga, x, z(4))),
            ("^rstd: shape", lambda: B.rms_backward(rp, x, ga, x, ga)), ("^dS: dtype", lambda: B.rms_backward(rp, x, ga, x, ga[:4], dS=x.float())),
            ("^S must be contiguous", lambda: B.rms_backward(rp, odd, ga, x, ga[:4])),
            ("^X must be contiguous", lambda: B.q8_pack(qp, odd)), ("^X: dtype", lambda: B.q8_pack(B.q8_plan(4, 16, B.MOE_F32), x)),
            ("^q: shape", lambda: B.q8_unpack(qp, q(4, 16), xs)), ("^s: shape", lambda: B.q8_unpack(qp, xq, s8(4, 1))),
            ("^q: dtype", lambda: B.q8_unpack(qp, z(4, 128, d=torch.uint8), xs)), ("^s: dtype", lambda: B.q8_unpack(qp, xq, z(4, 4, d=torch.uint8))),
            ("^along: 'M'", lambda: B.q8_pack_weights(w, "M")), ("^W: 2 dimensions", lambda: B.q8_pack_weights(x)),
            ("^unsupported dtype", lambda: B.q8_pack_weights(w.half())), ("^W must be contiguous", lambda: B.q8_pack_weights(z(2, 8, 16).transpose(1, 2))),
            ("^A: shape", lambda: B.q8_swiglu_forward(qp, x[:3], x)), ("^U: shape", lambda: B.q8_swiglu_forward(qp, x, x[:3])),
            ("^U: dtype", lambda: B.q8_swiglu_forward(qp, x, x.float())), ("^As: shape", lambda: B.q8_swiglu_backward(qp, (xq, s8(4, 3), xq, xs), x)),
            ("^Uq: dtype", lambda: B.q8_swiglu_backward(qp, (xq, xs, z(4, 128), xs), x)),
            ("^Us: shape", lambda: B.q8_swiglu_backward(qp, (xq, xs, xq, s8(4, 3)), x)), ("^dH: dtype", lambda: B.q8_swiglu_backward(qp, kept, x.float())),
            ("^offsets are required", lambda: B.gmm_forward(gp, x, w)), ("^offsets are required", lambda: B.gmm8_forward(g8, xq, xs, wq, ws)),
            ("^offsets: dtype", lambda: B.gmm_forward(gp, x, w, of.long())), ("^offsets: shape", lambda: B.gmm_backward_dx(gp, dy, w, of[:2])),
            ("^offsets: device", lambda: B.gmm_backward_dw(gp, x, dy, meta(of))), ("^offsets: shape", lambda: B.gmm8_backward_dw(g8, xq, xs, dy, of[:2])),
            ("^W: shape", lambda: B.gmm_forward(gp, x, z(2, 8, 16), of)), ("^W must be contiguous", lambda: B.gmm_forward(gp, x, z(2, 8, 16).transpose(1, 2), of)),
            ("^dY: shape", lambda: B.gmm_backward_dx(gp, x, w, of)), ("^W: dtype", lambda: B.gmm_backward_dx(gp, dy, w.float(), of)),
            ("^dY: shape", lambda: B.gmm_backward_dw(gp, x, x, of)), ("^X: dtype", lambda: B.gmm_backward_dw(gp, x.float(), dy, of)),
            ("^accumulate needs", lambda: B.gmm_backward_dw(gp, x, dy, of, accumulate=True)),
            ("^accumulate needs", lambda: B.gmm8_backward_dw(g8, xq, xs, dy, of, accumulate=True)),
            ("^Xq: shape", lambda: B.gmm8_forward(gp, xq, xs, wq, ws, of)), ("^Xs: shape", lambda: B.gmm8_forward(g8, xq, s8(4, 8), wq, ws, of)),
            ("^Wq: shape", lambda: B.gmm8_forward(g8, xq, xs, q(2, 16, 128), ws, of)), ("^Ws: shape", lambda: B.gmm8_forward(g8, xq, xs, wq, s8(2, 2, 4), of)),
            ("^Xq: dtype", lambda: B.gmm8_backward_dw(g8, z(4, 128), xs, dy, of)), ("^dY: shape", lambda: B.gmm8_backward_dw(g8, xq, xs, x, of))):
        with pytest.raises(ValueError, match=message):
            call()
    # and what passes every check is refused for its device alone
    for call in (lambda: B.rms_forward(rp, x, ga), lambda: B.rms_forward_q8(rp, x, ga, x), lambda: B.rms_backward(rp, x, ga, x, ga[:4], x),
                 lambda: B.q8_pack(qp, x), lambda: B.q8_unpack(qp, xq, xs), lambda: B.q8_pack_weights(w), lambda: B.q8_swiglu_forward(qp, x, x),
                 lambda: B.q8_swiglu_backward(qp, kept, x), lambda: B.gmm_forward(gp, x, w, of), lambda: B.gmm_backward_dx(gp, dy, w, of),
                 lambda: B.gmm_backward_dw(gp, x, dy, of), lambda: B.gmm8_forward(g8, xq, xs, wq, ws, of), lambda: B.gmm8_backward_dw(g8, xq, xs, dy, of)):
        with pytest.raises(ValueError, match="^tensors must be on a GPU, not on cpu$"):
            call()


def test_plans_ask_for_workspaces():
    """The sizes that test_gmm_workspaces goes through: which of them need one, so that its refusals are reached."""
    for name, (operands, _, _) in GMM.items():
        kind = "bwd_workspace_bytes" if name.endswith("dw") else "fwd_workspace_bytes"
        asked = [(R, K, E) for R in (1, 8, 64, 300, 5000) for K in (64, 2048, 16384) for E in (1, 4)
                 if getattr(B.gmm_plan(R, K, 2048, E, operands), kind) > 0]
        assert len(asked) >= 2, name
