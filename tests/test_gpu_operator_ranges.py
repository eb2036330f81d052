"""The operators at the ends of the float range, against their 64-bit definitions."""
import pytest
import torch

import ops_reference as ref
from test_gpu_adapters import _check as check_adapter, _ids, _inputs as adapter_inputs, _run as run_adapter

pytestmark = pytest.mark.gpu

TOP = 1.9921875 * 2.0 ** 127            # the largest bfloat16; a factor of 1.003 keeps it a finite float


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M", [8, 100])
@pytest.mark.parametrize("side", ["S", "P"])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_low_rank_activations_near_the_largest_float(dtype, M, side, sign):
    """scale down X (S), or scale up^T dY (P), past the largest bfloat16 and still a float: what is
    multiplied with it is small, so every output is finite."""
    t = adapter_inputs(dtype, M, 64, 48, 3, 4, bias=False)
    for name in ("x", "w", "a", "b", "dy"):
        t[name].zero_()
    t["x"][:, 0] = 1.0 if side == "S" else 2.0 ** -10
    t["dy"][:, 0] = 2.0 ** -10 if side == "S" else 1.0
    t["a"][:, 0, 0] = sign * TOP if side == "S" else 2.0 ** -20
    t["b"][:, 0, 0] = 2.0 ** -20 if side == "S" else sign * TOP
    t["scale"] = torch.tensor([1.003, 1.0, 1.0039])
    ids = _ids("mixed", M, 3)
    got = run_adapter(t, ids)
    assert all(torch.isfinite(v).all() for v in got.values())
    check_adapter(t, ids, got, side)
