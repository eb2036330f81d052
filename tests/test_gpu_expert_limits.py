"""The experts' operators at the ends of what they take: no experts at all, and products
of more workgroups than one dimension of a launch holds."""
import pytest
import torch

import experts_reference as xr
import ops_reference as ref
from test_gpu_experts import _check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,k", [(31, 2), (70, 2), (700, 3)])
@pytest.mark.parametrize("gate,bias", [(None, True), ("silu", True), ("gelu", False), ("relu", True)])
def test_no_experts(dtype, T, k, gate, bias):
    """Rows of no expert alone: outputs and gradients are zeros, whatever the number of rows."""
    _check(dtype, T, k, 0, 34, 40, gate, bias, "none")


def _wide_bank(dtype, n, N, K, used):
    """One row for each of n experts, and a bank that is zero but for the experts `used`."""
    from fp32_emulated_gemm_amd.experts import sort_tokens
    order = sort_tokens(torch.arange(n, dtype=torch.int32, device="cuda"), n)
    x = torch.randn(n, K, device="cuda").to(xr.DT[dtype])
    w = torch.zeros(n, N, K, dtype=x.dtype, device="cuda")
    for e in used:
        w[e] = torch.randn(N, K, device="cuda").to(x.dtype)
    return order, x, w


@pytest.mark.parametrize("dtype,n,N,K", [
    ("f32", 64, 2097200, 1),         # the kernel of few rows: 64 row tiles of 131075 workgroups of 512
    ("f32", 1024, 1048640, 1),       # 128 x 128 tiles: 1024 of 8193 and 512
    ("bf16", 1024, 1048640, 1),      # the same, of rows that do not lie in pieces
    ("bf16", 1024, 2097280, 8)])     # of rows that do, in tiles of any size
def test_forward_grids_of_more_than_32_bits(dtype, n, N, K):
    from fp32_emulated_gemm_amd.experts import expert_linear
    torch.manual_seed(N)
    used = (0, n // 2, n - 1)
    order, x, w = _wide_bank(dtype, n, N, K, used)
    h = expert_linear(x, w, order)
    rest = torch.ones(n, dtype=torch.bool)
    for e in used:
        want, mag = x[e].double() @ w[e].double().t(), x[e].double().abs() @ w[e].double().abs().t()
        # eight terms summed in 32 bits, one unit more for products left out, and the output's rounding
        tol = (2 * K + 2) * ref.U * mag + (ref.BF if dtype == "bf16" else 0.0) * want.abs() + ref.TINY
        assert bool(((h[e].double() - want).abs() <= tol).all()), e
        rest[e] = False
    assert all(not bool(h[e].any()) for e in rest.nonzero().flatten().tolist())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_backward_grids_of_more_than_32_bits(dtype):
    """dX and dW of 1024 experts of one row of 1048704 columns: products of one term."""
    from fp32_emulated_gemm_amd.experts import expert_linear
    n, K = 1024, 1048704
    order, x, w = _wide_bank(dtype, n, 1, K, (0, n - 1))
    x.requires_grad_(True), w.requires_grad_(True)
    dh = torch.randn(n, 1, device="cuda").to(x.dtype)
    dx, dw = torch.autograd.grad(expert_linear(x, w, order), (x, w), dh)
    for e in range(n):
        for got, operand in ((dx[e], w[e, 0]), (dw[e, 0], x[e])):
            want = dh[e, 0].double() * operand.detach().double()
            tol = 4 * ref.U * want.abs() + (ref.BF if dtype == "bf16" else 0.0) * want.abs() + ref.TINY
            assert bool(((got.double() - want).abs() <= tol).all()), e
