"""Arguments of the operators' tensor functions on the GPU: layouts of a weight."""
import pytest
import torch

import ops_reference as ref
from test_gpu_adapters import _ids, _inputs as adapter_inputs
from test_gpu_gated import _cuda, _inputs as gated_inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M", [8, 100])
@pytest.mark.parametrize("K", [64, 67])
def test_a_plan_of_the_other_operator_is_refused(dtype, M, K):
    """Also where the layouts agree (bfloat16 rows that are read as they lie, few rows)."""
    from fp32_emulated_gemm_amd import adapters, gated
    x, w, b, _ = (_cuda(t) for t in gated_inputs(dtype, M, K, 24, True))
    with pytest.raises(ValueError):
        gated.gated_linear(x, w, b, plan=adapters.plan_weight(w))
    ref.check(gated.gated_linear(x, w, b, plan=gated.plan_weight(w)), ref.gated(x.cpu(), w.cpu(), b.cpu(), "silu")["h"],
              "H")
    t = adapter_inputs(dtype, M, K, 48, 3, 4)
    c = {k: _cuda(v) for k, v in t.items()}
    ids = _ids("mixed", M, 3)
    for backward in (False, True):
        with pytest.raises(ValueError):
            adapters.adapter_linear(c["x"], c["w"], c["a"], c["b"], ids.cuda(), plan=gated.plan_weight(c["w"]))
        y = adapters.adapter_linear(c["x"], c["w"], c["a"], c["b"], ids.cuda(), c["scale"], c["bias"],
                                    plan=adapters.plan_weight(c["w"], backward=backward))
        ref.check(y, ref.adapter(t["x"], t["w"], t["a"], t["b"], ids, t["scale"], t["bias"])["y"], "Y")
