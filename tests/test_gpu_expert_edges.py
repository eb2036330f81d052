"""Experts and 4-bit banks where rows crowd one expert of many, and where values are not
finite in front of a gate."""
import pytest
import torch

import experts_reference as xr
import ops_reference as ref
from test_gpu_quant4 import _cuda, _pack, _products, _weights

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("T,k,n", [(450, 2, 64), (1024, 1, 64), (1025, 1, 64), (300, 3, 200)])
@pytest.mark.parametrize("kind", ["one", "few", "mixed"])
def test_crowded_banks(dtype, group, T, k, n, kind):
    """On both sides of the 16 rows an expert up to which the packed weights are read."""
    _products(dtype, T, k, n, 34, 200, group, True, "silu" if n == 200 else None, True, kind, seed=T)


def _bad_rows(x, seed):
    """One row with an Inf, one with a NaN, one with both signs of Inf."""
    P = x.shape[0]
    rows = sorted({0, P // 2, P - 1})
    for r, values in zip(rows, ((float("inf"),), (float("nan"),), (float("inf"), float("-inf")))):
        for i, v in enumerate(values):
            x[r, 3 + 5 * i] = v
    return rows


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("P", [3, 40, 300])
@pytest.mark.parametrize("gate", ["silu", "gelu", "gelu_tanh", "sigmoid", "relu"])
def test_rows_that_are_not_finite_before_a_gate(dtype, P, gate):
    """They reach the outputs and gradients of their own rows, and the weight gradient of their expert, alone;
    each of their outputs has an infinite or undefined factor."""
    from fp32_emulated_gemm_amd.experts import expert_linear, sort_tokens
    from fp32_emulated_gemm_amd.quant4 import quant4_linear
    n, N, K = 2, 48, 72
    g = torch.Generator().manual_seed(P)
    x = torch.randn(P, K, generator=g).to(xr.DT[dtype])
    w = (torch.randn(n, N, K, generator=g) * K ** -0.5).to(x.dtype)
    dh = torch.randn(P, N // 2, generator=g).to(x.dtype)
    ids = torch.zeros(P, 1, dtype=torch.int32)               # the other expert has no rows
    offsets, order = xr.order(ids, n)[0], sort_tokens(ids.cuda(), n)
    clean = xr.experts(x, w, offsets, None, gate, dh)
    dirty = x.clone()
    rows = _bad_rows(dirty, P)
    rest = torch.ones(P, dtype=torch.bool)
    rest[rows] = False
    xd, wd = dirty.cuda().requires_grad_(True), w.cuda().requires_grad_(True)
    h = expert_linear(xd, wd, order, gate=gate)
    dx, dw = torch.autograd.grad(h, (xd, wd), dh.cuda())
    assert not bool(h[rows].isfinite().any())
    for got, name in ((h, "h"), (dx, "dx")):
        want, bound = clean[name]
        ref.check(got.detach().cpu()[rest], (want[rest], bound[rest]), name)
    assert not bool(dw[1].any()) and bool(dw[0].isnan().any())

    q, scale, zero = _weights(n, N, K, 32, True, P)
    w4 = _pack(q, scale, _cuda(zero), 32, True)
    few = P <= 64
    h = quant4_linear(dirty.cuda(), w4, gate=gate, order=order).cpu()
    want, bound = xr.quant4(x, q, scale, zero, 32, offsets, None, gate, few)
    assert not bool(h[rows].isfinite().any())
    ref.check(h[rest], (want[rest], bound[rest]), "4 bits")
