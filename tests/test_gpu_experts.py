"""The experts' products on sorted rows, forward and backward, against the 64-bit
definition at derived bounds."""
import pytest
import torch

import experts_reference as xr
import ops_reference as ref

pytestmark = pytest.mark.gpu


def _inputs(dtype, P, N, K, n, gate, bias, seed=0):
    g = torch.Generator().manual_seed(seed)

    def normal(*shape, sigma=1.0):
        return (torch.randn(shape, generator=g) * sigma).to(xr.DT[dtype])

    return (normal(P, K), normal(n, N, K, sigma=max(K, 1) ** -0.5), normal(n, N, sigma=0.1) if bias else None,
            normal(P, N // 2 if gate else N))


def _check(dtype, T, k, n, N, K, gate, bias, kind, seed=0):
    from fp32_emulated_gemm_amd.experts import expert_linear, sort_tokens
    ids = xr.make_ids(kind, T, k, n, seed)
    offsets = xr.order(ids, n)[0]
    order = sort_tokens(ids.cuda(), n)
    x, w, b, dh = _inputs(dtype, T * k, N, K, n, gate, bias, seed)
    x[offsets[-1]:], dh[offsets[-1]:] = float("nan"), float("nan")     # rows of no expert
    want = xr.experts(x, w, offsets, b, gate, dh)
    leaves = [t.cuda().requires_grad_(True) for t in (x, w, b) if t is not None]
    xd, wd, bd = leaves[0], leaves[1], leaves[2] if bias else None
    h = expert_linear(xd, wd, order, bd, gate)
    grads = torch.autograd.grad(h, leaves, dh.cuda())
    ref.check(h.detach(), want["h"], "h")
    for got, name in zip(grads, ("dx", "dw", "db")):
        ref.check(got, want[name], name)
    with torch.no_grad():
        ref.check(expert_linear(xd, wd, order, bd, gate), want["h"], "h without gradients")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,k,n,N,K", [
    (1, 1, 1, 2, 1), (1, 2, 8, 64, 64), (5, 2, 3, 34, 33), (16, 2, 32, 96, 128), (40, 3, 4, 130, 257), (64, 1, 1, 128, 100),
    (200, 2, 5, 96, 64), (300, 2, 3, 256, 320), (129, 4, 2, 262, 65), (700, 2, 9, 66, 40)])
@pytest.mark.parametrize("gate,bias", [(None, True), ("silu", False), ("gelu", True)])
def test_products(dtype, T, k, n, N, K, gate, bias):
    _check(dtype, T, k, n, N, K, gate, bias, "mixed", seed=T)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["one", "none", "few", "full"])
@pytest.mark.parametrize("T", [9, 130])
def test_experts_without_rows(dtype, kind, T):
    _check(dtype, T, 2, 5, 64, 48, "silu", True, kind)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("gate", ["gelu_tanh", "sigmoid", "relu"])
def test_other_gates(dtype, gate):
    _check(dtype, 50, 2, 3, 48, 40, gate, True, "mixed")
    _check(dtype, 3, 2, 3, 48, 40, gate, True, "mixed")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,k,n,N,K", [(0, 2, 3, 8, 8), (4, 2, 3, 0, 8), (4, 2, 3, 8, 0), (4, 0, 3, 8, 8), (4, 2, 0, 8, 8),
                                       (70, 2, 3, 8, 0)])
@pytest.mark.parametrize("gate", [None, "silu"])
def test_empty(dtype, T, k, n, N, K, gate):
    _check(dtype, T, k, n, N, K, gate, True, "none" if n == 0 else "mixed")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [20, 700])
def test_values_that_are_not_finite_stay_in_their_rows(dtype, T):
    """Inf and NaN in one expert's weights and in one row of X reach the outputs and gradients of those
    alone, and make them Inf or NaN."""
    from fp32_emulated_gemm_amd.experts import expert_linear, sort_tokens
    n, N, K = 3, 40, 72
    ids = (torch.arange(T) % n).int().unsqueeze(1)
    offsets = xr.order(ids, n)[0].tolist()
    order = sort_tokens(ids.cuda(), n)
    x, w, _, dh = _inputs(dtype, T, N, K, n, None, False)
    clean = xr.experts(x, w, torch.tensor(offsets), None, None, dh)
    w[1, 7, 5] = float("inf")
    x[offsets[3] - 1, 9] = float("-inf")
    x[0, 3] = float("nan")
    xd, wd = x.cuda().requires_grad_(True), w.cuda().requires_grad_(True)
    h = expert_linear(xd, wd, order)
    dx, dw = torch.autograd.grad(h, (xd, wd), dh.cuda())
    h, dx, dw = h.detach().cpu(), dx.cpu(), dw.cpu()
    s, t = offsets[1], offsets[2]
    rows = torch.ones(T, dtype=torch.bool)
    rows[0] = rows[-1] = False
    assert h[0].isnan().all() and not h[-1].isfinite().any() and not h[s:t, 7].isfinite().any()
    ok = rows.unsqueeze(1).expand(T, N).clone()
    ok[s:t, 7] = False
    bad = (h.double() - clean["h"][0]).abs() > clean["h"][1]
    assert not (bad & ok).any()
    other = torch.cat((torch.arange(s), torch.arange(t, T)))
    assert ((dx.double() - clean["dx"][0]).abs() <= clean["dx"][1])[other].all()
    assert ((dw.double() - clean["dw"][0]).abs() <= clean["dw"][1])[1].all()
