"""Checks of the operators' arguments that need no GPU: what the tensor functions
make of strides, and which layouts of a weight they take."""
import pytest
import torch


@pytest.mark.parametrize("held", [None, "laid out"])
def test_a_plan_stands_for_its_own_operator_only(held):
    """The two layouts have one shape and type, whether the forward's rows are copied or lie."""
    from fp32_emulated_gemm_amd.ops import WeightPlan
    w = torch.zeros(6, 8)
    for gated in (True, False):
        plan = WeightPlan.__new__(WeightPlan)
        plan.dtype, plan.shape, plan.device, plan.gated = w.dtype, (6, 8), w.device, gated
        plan.forward, plan.backward = held, None
        plan.check(w, gated=gated)
        with pytest.raises(ValueError):
            plan.check(w, gated=not gated)
        with pytest.raises(ValueError):
            plan.check(w[:4], gated=gated)
