"""The operators at the ends of the float range, against their 64-bit definitions."""
import pytest
import torch

import ops_reference as ref
from test_gpu_adapters import _check as check_adapter, _ids, _inputs as adapter_inputs, _run as run_adapter
from test_gpu_gated import _run as run_gated

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


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("gate", ["silu", "gelu", "gelu_tanh", "sigmoid", "relu"])
def test_large_gate_values_have_gradients(dtype, gate):
    """Gate values of +-2^0 .. +-2^100, whose squares are no floats: the activation's derivative is 0
    or 1 from 2^6 on."""
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    M, K, F = 70, 8, 202
    x, w, dh = torch.zeros(M, K), torch.zeros(2 * F, K), torch.full((M, F), 2.0 ** -60)
    x[:, 0] = 2.0 ** -20
    exponent = torch.arange(F) // 2
    w[:F, 0] = 2.0 ** (20.0 + exponent) * (1 - 2 * (torch.arange(F) % 2))
    w[F:, 0] = 2.0 ** 20
    x, w, dh = x.to(dt), w.to(dt), dh.to(dt)
    want = ref.gated(x, w, None, gate, dh)
    got = run_gated(x, w, None, dh, gate)
    for name in ("h0", "h", "dx", "dw"):
        assert torch.isfinite(got[name]).all(), name
        ref.check(got[name], want[name.rstrip("0")], name)
    # dW's gate rows are M dh act'(z) x (up = 1): a power of two near 70, or zero
    far = got["dw"][:F, 0].double().cpu()[12:]
    slope = torch.zeros_like(far) if gate == "sigmoid" else (torch.arange(F - 12) % 2 == 0).double()
    full = M * 2.0 ** -80
    assert ((far - slope * full).abs() <= 2.0 ** -8 * full).all()
