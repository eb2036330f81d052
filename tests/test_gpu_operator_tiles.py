"""The operators' bfloat16 products at the sizes that take each of their tiles,
and the launches that leave the last rows or columns to smaller tiles."""
import pytest
import torch

import ops_reference as ref
from test_gpu_adapters import _check as check_adapter, _ids, _inputs as adapter_inputs, _run as run_adapter
from test_gpu_gated import _cuda, _inputs as gated_inputs

pytestmark = pytest.mark.gpu

# M, K, outputs of the product
SHAPES = [(1000, 512, 4006), (2040, 256, 4082), (4090, 192, 4094), (4608, 512, 4096), (8180, 256, 2120)]


@pytest.mark.parametrize("M,K,N", SHAPES)
def test_gated(M, K, N):
    from fp32_emulated_gemm_amd.gated import gated_linear
    x, w, b, _ = gated_inputs("bf16", M, K, N // 2, True, seed=M)
    ref.check(gated_linear(_cuda(x), _cuda(w), _cuda(b)), ref.gated(x, w, b, "silu")["h"], "H")


@pytest.mark.parametrize("M,K,N", [(4608, 200, 136), (2500, 4096, 40)])
def test_gated_gradients(M, K, N):
    """A long sum over the rows in the weight's gradient, in K slices."""
    from fp32_emulated_gemm_amd.gated import gated_linear
    x, w, _, dh = gated_inputs("bf16", M, K, N // 2, False, seed=M)
    want = ref.gated(x, w, None, "silu", dh)
    xs, ws = _cuda(x).requires_grad_(True), _cuda(w).requires_grad_(True)
    dx, dw = torch.autograd.grad(gated_linear(xs, ws), (xs, ws), dh.cuda())
    ref.check(dx, want["dx"], "dx")
    ref.check(dw, want["dw"], "dw")


@pytest.mark.parametrize("M,K,N", SHAPES)
@pytest.mark.parametrize("r", [6, 5])
def test_adapters(M, K, N, r):
    t = adapter_inputs("bf16", M, K, N, 4, r, seed=M)
    ids = _ids("spans" if r == 6 else "mixed", M, 4)
    got = run_adapter(t, ids)
    check_adapter(t, ids, got, f"{M}x{K}x{N}")


def test_ranks_past_an_even_rank_stay_out():
    """A rank of 6 ends inside a 16-byte piece: the next row of the up factor holds
    infinities, which belong to that output alone."""
    t = adapter_inputs("bf16", 200, 64, 96, 2, 6, seed=5)
    t["b"][:, 1::2, :] = float("inf")
    from fp32_emulated_gemm_amd.adapters import adapter_linear
    c = {k: _cuda(v) for k, v in t.items()}
    ids = torch.arange(200, dtype=torch.int32).cuda() % 2
    y = adapter_linear(c["x"], c["w"], c["a"], c["b"], ids, c["scale"], c["bias"])
    assert torch.isfinite(y[:, ::2]).all()
    assert not torch.isfinite(y[:, 1::2]).any()
