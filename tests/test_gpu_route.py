"""Tokens sorted by expert and back: the order bit for bit, rows moved, gradients
against the 64-bit definition."""
import pytest
import torch

import experts_reference as xr
import ops_reference as ref

pytestmark = pytest.mark.gpu


def _values(shape, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g).to(xr.DT[dtype])


def _same_order(order, ids, n):
    for got, want, name in zip((order.offsets, order.pairs, order.places), xr.order(ids, n),
                               ("offsets", "pairs", "places")):
        assert got.dtype == torch.int32 and torch.equal(got.cpu(), want), name


@pytest.mark.parametrize("T,k,n", [(0, 2, 4), (1, 1, 1), (1, 8, 64), (5, 3, 7), (16, 2, 1024), (333, 3, 1023), (1024, 4, 64),
                                   (4096, 1, 5), (4097, 1, 5), (1366, 3, 128), (20001, 2, 60), (9000, 8, 1024), (7, 2, 0)])
@pytest.mark.parametrize("kind", ["mixed", "full", "one", "none", "few"])
def test_order(T, k, n, kind):
    from fp32_emulated_gemm_amd.experts import sort_tokens
    if n == 0 and kind in ("one", "few"):
        pytest.skip("no expert to take")
    ids = xr.make_ids(kind, T, k, n, seed=T + n)
    _same_order(sort_tokens(ids.cuda(), n), ids, n)


def test_order_of_other_layouts():
    """One dimension; columns of a wider tensor; a transposed one."""
    from fp32_emulated_gemm_amd.experts import sort_tokens
    ids = xr.make_ids("mixed", 100, 6, 9)
    _same_order(sort_tokens(ids[:, 2:4].cuda(), 9), ids[:, 2:4], 9)
    _same_order(sort_tokens(ids.cuda()[:, 1:6:2], 9), ids[:, 1:6:2], 9)
    _same_order(sort_tokens(ids.cuda().t(), 9), ids.t(), 9)
    order = sort_tokens(ids[:, 0].cuda(), 9)
    assert (order.tokens, order.choices) == (100, 1)
    _same_order(order, ids[:, :1], 9)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,k,n,K", [(1, 1, 1, 1), (1, 4, 8, 4096), (5, 3, 7, 3), (64, 2, 16, 1030), (257, 5, 33, 512),
                                     (100, 8, 4, 2044), (3, 2, 2, 0), (0, 2, 2, 8), (4, 0, 2, 8)])
@pytest.mark.parametrize("kind", ["mixed", "one", "none"])
def test_rows_there_and_back(dtype, T, k, n, K, kind):
    from fp32_emulated_gemm_amd.experts import combine_tokens, gather_tokens, sort_tokens
    ids = xr.make_ids(kind, T, k, n, seed=K)
    offsets, pairs, places = xr.order(ids, n)
    order = sort_tokens(ids.cuda(), n)
    x = _values((T, K), dtype, 1)
    leaf = x.cuda().requires_grad_(True)
    xs = gather_tokens(leaf, order)
    want = torch.where((pairs >= 0).unsqueeze(1), x[pairs.long().clamp(min=0) // max(k, 1)] if T else x, 0)
    assert torch.equal(xs.detach().cpu(), want.to(x.dtype))
    dxs = _values((T * k, K), dtype, 2)
    dxs[offsets[-1]:] = float("nan")            # rows of no expert
    dx, = torch.autograd.grad(xs, (leaf,), dxs.cuda())
    ref.check(dx, xr.combine(dxs, places, None)["y"], "dx")

    ys, dy = _values((T * k, K), dtype, 3), _values((T, K), dtype, 4)
    ys[offsets[-1]:] = float("nan")
    weights = torch.rand(T, k, generator=torch.Generator().manual_seed(5)) - 0.25
    for w in (weights, None):
        a, b = ys.cuda().requires_grad_(True), None if w is None else w.cuda().requires_grad_(True)
        y = combine_tokens(a, order, b)
        want = xr.combine(ys, places, w, dy)
        ref.check(y.detach(), want["y"], "y")
        grads = torch.autograd.grad(y, (a,) if w is None else (a, b), dy.cuda())
        ref.check(grads[0], want["dys"], "dys")
        if w is not None:
            ref.check(grads[1], want["dw"], "dweights")
            only, = torch.autograd.grad(combine_tokens(ys.cuda(), order, b), (b,), dy.cuda())
            assert torch.equal(only, grads[1])
    with torch.no_grad():
        assert torch.equal(combine_tokens(ys.cuda(), order, weights.cuda()),
                           combine_tokens(a.detach(), order, weights.cuda()))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_strides(dtype):
    """Rows of wider tensors at odd offsets, transposed and expanded tensors, on both sides."""
    from fp32_emulated_gemm_amd.experts import combine_tokens, gather_tokens, sort_tokens
    T, k, n, K = 33, 3, 5, 70
    ids = xr.make_ids("mixed", T, k, n)
    order, places = sort_tokens(ids.cuda(), n), xr.order(ids, n)[2]
    wide = _values((T, K + 9), dtype, 1).cuda()
    tall = _values((T * k, K + 5), dtype, 2).cuda()
    across = _values((K, T), dtype, 3).cuda()
    weights = torch.rand(k, T).cuda().t()
    for x in (wide[:, 1:K + 1], wide[:, 8:K + 8], across.t(), wide[:1, :K].expand(T, K)):
        assert torch.equal(gather_tokens(x, order), gather_tokens(x.contiguous(), order))
    for ys in (tall[:, 3:K + 3], tall[:, :K], tall[:1, :K].expand(T * k, K)):
        ref.check(combine_tokens(ys, order, weights), xr.combine(ys.cpu(), places, weights.cpu())["y"], "y")
    leaf = tall[:, 3:K + 3].detach().requires_grad_(True)
    dy = across.t()
    grad, = torch.autograd.grad(combine_tokens(leaf, order, weights), (leaf,), dy)
    ref.check(grad, xr.combine(leaf.detach().cpu(), places, weights.cpu(), dy.cpu())["dys"], "dys")


def test_places_outside_the_rows_lead_nowhere():
    """Corrupt arrays: nothing is read or written outside the operands."""
    from fp32_emulated_gemm_amd.experts import ExpertOrder, combine_tokens, gather_tokens
    T, k, K = 6, 2, 40
    places = torch.tensor([[0, 12], [-5, 3], [1 << 30, 4], [5, -(1 << 31)], [11, 6], [7, 100]], dtype=torch.int32)
    for last in (-7, 5, 12, 1 << 30):
        offsets = torch.tensor([0, 3, last], dtype=torch.int32).cuda()
        order = ExpertOrder(offsets, torch.zeros(12, dtype=torch.int32).cuda(), places.cuda(), 2)
        x = _values((T, K), "f32", 1)
        xs = gather_tokens(x.cuda(), order).cpu()
        rest = max(last, 0)
        for t in range(T):
            for j in range(k):
                if 0 <= places[t, j] < min(12, rest):
                    assert torch.equal(xs[places[t, j]], x[t])
        inside = torch.where((places >= 0) & (places < 12), places, -1)
        ref.check(combine_tokens(xs.cuda(), order), xr.combine(xs, inside, None)["y"], "y")
