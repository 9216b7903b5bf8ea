"""The tensors that the binding makes for outputs: what torch.empty would have made, in every mode that changes that."""

import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

from gpu_common import DEV, B, needs_gpu, require_lib

pytestmark = [pytest.mark.gpu, needs_gpu]


def calls():
    """One call of every operator family, from the same inputs: its outputs."""
    g = torch.Generator().manual_seed(0)
    r = lambda *s: torch.randn(*s, generator=g).bfloat16().to(DEV)
    x, gamma, w = r(9, 40), torch.ones(40, device=DEV), r(2, 40, 24)
    out = list(B.lnorm_forward(B.lnorm_plan(9, 40), x, gamma, gamma))
    out += B.rms_forward(B.rms_plan(9, 40), x, gamma, x)
    q, s, *_ = B.rms_forward_q8(B.rms_plan(9, 40), x, gamma)
    out += [q.view(torch.uint8), s.view(torch.uint8)]
    off = torch.tensor([0, 3, 9], dtype=torch.int32, device=DEV)
    plan = B.gmm_plan(9, 40, 24, 2)
    y = B.gmm_forward(plan, x, w, off)
    out += [y, B.gmm_backward_dx(plan, y, w, off), B.gmm_backward_dw(plan, x, y, off)]
    hq, hs, kept = B.q8_swiglu_forward(B.q8_plan(9, 24), y, y)
    out += [hq.view(torch.uint8), hs.view(torch.uint8), *B.q8_swiglu_backward(B.q8_plan(9, 24), kept, y)]
    return out


def test_outputs_are_whole_tensors():
    require_lib()
    for t in calls():
        assert t.is_contiguous() and t.device == DEV and not t.requires_grad and t.untyped_storage().nbytes() >= t.nbytes


def test_outputs_without_the_direct_allocation(monkeypatch):
    """Where this torch has no such call, through torch.empty: the same bits."""
    want = calls()
    monkeypatch.setattr(B, "_empty_strided", None)
    for a, b in zip(want, calls()):
        assert torch.equal(a, b) and a.stride() == b.stride()


def test_deterministic_mode_fills_what_a_call_leaves():
    """Rows of no expert are left as they are: under deterministic algorithms torch.empty makes them NaN."""
    x, w = torch.ones(50, 16, device=DEV).bfloat16(), torch.ones(1, 16, 8, device=DEV).bfloat16()
    off = torch.tensor([0, 3], dtype=torch.int32, device=DEV)
    plan = B.gmm_plan(50, 16, 8, 1)
    junk = [torch.zeros(50, 8, device=DEV).bfloat16() for _ in range(8)]  # what new memory held last
    del junk
    torch.use_deterministic_algorithms(True)
    try:
        y = B.gmm_forward(plan, x, w, off)
    finally:
        torch.use_deterministic_algorithms(False)
    assert bool((y[:3] == 16).all()) and torch.isnan(y[3:]).all()


def test_dispatch_modes_see_the_outputs():
    class Seen(TorchDispatchMode):
        made = 0

        def __torch_dispatch__(self, func, types, args=(), kwargs=None):
            out = func(*args, **(kwargs or {}))
            self.made += func.overloadpacket in (torch.ops.aten.empty, torch.ops.aten.empty_strided)
            return out

    x, gamma = torch.ones(9, 40, device=DEV).bfloat16(), torch.ones(40, device=DEV)
    plan = B.rms_plan(9, 40)
    with Seen() as seen:
        B.rms_forward(plan, x, gamma, x)  # Y, S, rstd
    assert seen.made == 3


def test_inference_mode():
    with torch.inference_mode():
        assert all(t.is_inference() for t in calls())
