"""Arguments of the operators' tensor functions on the GPU: layouts of a weight, rows far
apart, tangents, empty inputs of more dimensions."""
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


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_last_tokens_of_long_prompts(dtype):
    """One row, or several, of a buffer whose sequences lie further apart than a leading dimension
    may: inputs, weights and output gradients alike."""
    from fp32_emulated_gemm_amd.adapters import adapter_linear
    from fp32_emulated_gemm_amd.gated import gated_linear
    K, F, step = 64, 16, 8_388_544 + 64
    for M in (1, 2, 3):
        x, w, b, dh = gated_inputs(dtype, M, K, F, True, seed=M)
        hidden = torch.zeros(M, step // K, K, dtype=x.dtype, device="cuda")
        xs = hidden[:, -1]
        xs.copy_(x)
        grads = torch.zeros(M, step, dtype=x.dtype, device="cuda")[:, 8:8 + F]
        grads.copy_(dh)
        want = ref.gated(x, w, b, "silu", dh)
        ref.check(gated_linear(xs, w.cuda(), b.cuda()), want["h"], "H")
        leaf = xs.detach().requires_grad_(True)
        dx, = torch.autograd.grad(gated_linear(leaf, w.cuda(), b.cuda()), (leaf,), grads)
        ref.check(dx, want["dx"], "dx")
        t = adapter_inputs(dtype, M, K, F, 2, 4, seed=M)
        c = {k: _cuda(v) for k, v in t.items()}
        ids = torch.arange(M, dtype=torch.int32) % 2
        xs.copy_(t["x"])
        grads.copy_(t["dy"])
        want = ref.adapter(t["x"], t["w"], t["a"], t["b"], ids, t["scale"], t["bias"], t["dy"])
        leaf = xs.detach().requires_grad_(True)
        y = adapter_linear(leaf, c["w"], c["a"], c["b"], ids.cuda(), c["scale"], c["bias"])
        ref.check(y.detach(), want["y"], "Y")
        ref.check(torch.autograd.grad(y, (leaf,), grads)[0], want["dx"], "dx")
        wide = torch.zeros(F, step, dtype=x.dtype, device="cuda")[:, :K]
        wide.copy_(t["w"])
        y = adapter_linear(xs, wide, c["a"], c["b"], ids.cuda(), c["scale"], c["bias"])
        ref.check(y, want["y"], "Y, rows of W far apart")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M", [8, 100])
@pytest.mark.parametrize("grad", [True, False])
def test_tangents_are_refused(dtype, M, grad):
    """Forward-mode derivatives are not provided: an operand with a tangent raises, and none is
    dropped; without one, a call inside an open level computes as ever."""
    from torch.autograd import forward_ad
    from fp32_emulated_gemm_amd.adapters import adapter_linear
    from fp32_emulated_gemm_amd.gated import gated_linear
    x, w, b, _ = (_cuda(t) for t in gated_inputs(dtype, M, 64, 24, True))
    c = {k: _cuda(v) for k, v in adapter_inputs(dtype, M, 64, 48, 3, 4).items()}
    ids = _ids("mixed", M, 3).cuda()
    names = ("x", "w", "a", "b", "scale", "bias")

    def adapters(t):
        return adapter_linear(t["x"], t["w"], t["a"], t["b"], ids, t["scale"], t["bias"])

    with torch.set_grad_enabled(grad):
        with forward_ad.dual_level():
            for k in range(3):
                t = [x, w, b]
                t[k] = forward_ad.make_dual(t[k], torch.ones_like(t[k]))
                with pytest.raises(NotImplementedError):
                    gated_linear(*t)
            for name in names:
                t = dict(c)
                t[name] = forward_ad.make_dual(t[name], torch.ones_like(t[name]))
                with pytest.raises(NotImplementedError):
                    adapters(t)
            h, y = gated_linear(x, w, b), adapters(c)
        ref.check(h, ref.gated(x.cpu(), w.cpu(), b.cpu(), "silu")["h"], "H")
        t = {k: v.cpu() for k, v in c.items()}
        ref.check(y, ref.adapter(t["x"], t["w"], t["a"], t["b"], ids.cpu(), t["scale"], t["bias"])["y"], "Y")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lead", [(2, 3), (2, 50), (0, 3), ()])
@pytest.mark.parametrize("K", [0, 8])
def test_leading_dimensions_keep_the_graph(dtype, lead, K):
    """Any number of leading dimensions, empty ones and an empty K among them, has a gradient."""
    from fp32_emulated_gemm_amd.adapters import adapter_linear
    from fp32_emulated_gemm_amd.gated import gated_linear
    M = torch.Size(lead).numel()
    x, w, b, dh = gated_inputs(dtype, M, K, 6, True)
    leaf = x.cuda().reshape(*lead, K).requires_grad_(True)
    h = gated_linear(leaf, w.cuda(), b.cuda())
    assert h.shape == (*lead, 6)
    dx, = torch.autograd.grad(h, (leaf,), dh.cuda().reshape(*lead, 6))
    want = ref.gated(x, w, b, "silu", dh)
    ref.check(h.detach().reshape(M, 6), want["h"], "H")
    ref.check(dx.reshape(M, K), want["dx"], "dx")
    t = adapter_inputs(dtype, M, K, 6, 2, 4)
    c = {k: _cuda(v) for k, v in t.items()}
    ids = torch.arange(M, dtype=torch.int32) % 2
    leaf = c["x"].reshape(*lead, K).requires_grad_(True)
    y = adapter_linear(leaf, c["w"], c["a"], c["b"], ids.cuda().reshape(lead), c["scale"], c["bias"])
    dx, = torch.autograd.grad(y, (leaf,), c["dy"].reshape(*lead, 6))
    want = ref.adapter(t["x"], t["w"], t["a"], t["b"], ids, t["scale"], t["bias"], t["dy"])
    ref.check(y.detach().reshape(M, 6), want["y"], "Y")
    ref.check(dx.reshape(M, K), want["dx"], "dx")
