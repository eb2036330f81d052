"""What the experts' operators hold for their backward passes: operands that the gradients asked
for do not read may change in between, and are not kept."""
import pytest
import torch

import experts_reference as xr

pytestmark = pytest.mark.gpu


def _operands(dtype, gate=None, seed=0):
    from fp32_emulated_gemm_amd.experts import sort_tokens
    g = torch.Generator("cuda").manual_seed(seed)
    T, k, n, N, K = 50, 2, 3, 48, 40
    order = sort_tokens(torch.randint(-1, n, (T, k), generator=g, device="cuda", dtype=torch.int32), n)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda").to(xr.DT[dtype])

    return order, normal(T * k, K), normal(n, N, K), normal(n, N), normal(T * k, N // 2 if gate else N), normal(T, K)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("weighted", [False, True])
def test_rows_of_combine_may_change(dtype, weighted):
    from fp32_emulated_gemm_amd.experts import combine_tokens
    order, ys, _, _, _, dy = _operands(dtype)
    weights = torch.rand(50, 2, device="cuda") if weighted else None
    leaf = ys.clone().requires_grad_(True)
    want, = torch.autograd.grad(combine_tokens(leaf, order, weights), (leaf,), dy)
    rows = leaf * 1
    y = combine_tokens(rows, order, weights)
    rows.detach().fill_(7.0)
    got, = torch.autograd.grad(y, (leaf,), dy)
    assert torch.equal(got, want)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("gate", [None, "silu"])
def test_operands_of_products_may_change(dtype, gate):
    """The rows where the weight is fixed, the weight where the rows are, both where only a bias is trained."""
    from fp32_emulated_gemm_amd.experts import expert_linear
    order, x, w, b, dh, _ = _operands(dtype, gate)
    for trained, change in ((("x", "b"), "x"), (("w", "b"), "w"), (("b",), "xw"), (("x", "w", "b"), "")):
        t = {"x": x.clone(), "w": w.clone(), "b": b.clone()}
        leaves = [t[name].requires_grad_(True) for name in trained]
        want = torch.autograd.grad(expert_linear(t["x"], t["w"], order, t["b"], gate), leaves, dh)
        held = {name: v * 1 for name, v in t.items()}
        h = expert_linear(held["x"], held["w"], order, held["b"], gate)
        for name in change:
            held[name].detach().fill_(7.0)
        for a, c in zip(torch.autograd.grad(h, leaves, dh), want):
            assert torch.equal(a, c), (trained, change)


def test_a_needed_operand_that_changed_is_refused():
    from fp32_emulated_gemm_amd.experts import combine_tokens, expert_linear
    order, x, w, _, dh, dy = _operands("f32")
    weights = torch.rand(50, 2, device="cuda", requires_grad=True)
    rows = x.clone()
    y = combine_tokens(rows, order, weights)
    rows.fill_(7.0)
    with pytest.raises(RuntimeError):
        torch.autograd.grad(y, (weights,), dy)
    leaf, held = x.clone().requires_grad_(True), w.clone()
    h = expert_linear(leaf, held, order)
    held.fill_(7.0)
    with pytest.raises(RuntimeError):
        torch.autograd.grad(h, (leaf,), dh)
