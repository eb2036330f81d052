"""Modules with fixed weights on the GPU: what they compute follows the weight, however
it was written, and copies of a module compute what the module does."""
import copy

import pytest
import torch

import ops_reference as ref
from test_gpu_adapters import _ids

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def _half(m):
    m.weight.data.mul_(0.5)


def _assign(m):
    m.weight.data = m.weight.data * 0.5


def _twice(m):
    """Two assignments: the second may land where the fixed weight lay."""
    _assign(m)
    _assign(m)


def _vector(m):
    flat = torch.nn.utils.parameters_to_vector([m.weight]) * 0.5
    torch.nn.utils.vector_to_parameters(flat, [m.weight])


def _away(m):
    m.cpu()
    m.weight.data.mul_(0.5)
    m.cuda()


WRITES = [_half, _assign, _twice, _vector, _away]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows", [9, 100])
@pytest.mark.parametrize("write", WRITES)
def test_writes_that_torch_does_not_count(dtype, rows, write):
    from fp32_emulated_gemm_amd.adapters import AdapterLinear
    from fp32_emulated_gemm_amd.gated import GatedLinear
    torch.manual_seed(3)
    x, ids = torch.randn(rows, 72, device="cuda").to(DT[dtype]), _ids("mixed", rows, 3)
    m = GatedLinear(72, 40, device="cuda", dtype=DT[dtype]).fix_weights()
    m(x)
    write(m)
    want = ref.gated(x.cpu(), m.weight.detach().cpu(), m.bias.detach().cpu(), "silu")["h"]
    ref.check(m(x), want, "GatedLinear")

    m = AdapterLinear(72, 40, 3, 4, device="cuda", dtype=DT[dtype])
    with torch.no_grad():
        m.up.normal_()
    m.fix_weights()
    dy = torch.randn(rows, 40, device="cuda").to(DT[dtype])
    leaf = x.clone().requires_grad_(True)
    torch.autograd.grad(m(leaf, ids.cuda()), (leaf,), dy)
    write(m)
    t = [v.detach().cpu() for v in (m.weight, m.down, m.up)]
    want = ref.adapter(x.cpu(), *t, ids, m.scale.cpu(), m.bias.detach().cpu(), dy.cpu())
    y = m(leaf, ids.cuda())
    ref.check(y.detach(), want["y"], "AdapterLinear")
    ref.check(torch.autograd.grad(y, (leaf,), dy)[0], want["dx"], "AdapterLinear dx")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_copies_and_a_caller_s_plan(dtype):
    from fp32_emulated_gemm_amd import adapters, gated
    torch.manual_seed(5)
    x, ids = torch.randn(100, 67, device="cuda").to(DT[dtype]), _ids("mixed", 100, 3).cuda()
    m = gated.GatedLinear(67, 40, device="cuda", dtype=DT[dtype]).fix_weights()
    want = m(x)
    assert torch.equal(copy.deepcopy(m)(x), want)
    assert torch.equal(m(x, plan=gated.plan_weight(m.weight)), want)
    with pytest.raises(ValueError):
        m(x, plan=adapters.plan_weight(m.weight))
    m = adapters.AdapterLinear.from_linear(torch.nn.Linear(67, 40, device="cuda", dtype=DT[dtype]), 3, 4)
    with torch.no_grad():
        m.up.normal_()
        want = m(x, ids)
        assert torch.equal(copy.deepcopy(m)(x, ids), want)
        assert torch.equal(m(x, ids, plan=adapters.plan_weight(m.weight, backward=True)), want)
    with torch.no_grad():
        m.weight.mul_(2)
    with pytest.raises(RuntimeError):
        m(x, ids)
    with pytest.raises(RuntimeError):
        copy.deepcopy(m)(x, ids)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows", [9, 100])
def test_modules_made_and_run_for_inference(dtype, rows):
    from fp32_emulated_gemm_amd.adapters import AdapterLinear
    from fp32_emulated_gemm_amd.gated import GatedLinear
    torch.manual_seed(7)
    with torch.inference_mode():
        x, ids = torch.randn(rows, 72, device="cuda").to(DT[dtype]), _ids("mixed", rows, 3)
        m = GatedLinear(72, 40, device="cuda", dtype=DT[dtype]).fix_weights()
        ref.check(m(x), ref.gated(x.cpu(), m.weight.cpu(), m.bias.cpu(), "silu")["h"], "GatedLinear")
        m = AdapterLinear.from_linear(torch.nn.Linear(72, 40, device="cuda", dtype=DT[dtype]), 3, 4)
        m.up.normal_()
        t = [v.cpu() for v in (m.weight, m.down, m.up)]
        ref.check(m(x, ids.cuda()), ref.adapter(x.cpu(), *t, ids, m.scale.cpu(), m.bias.cpu())["y"], "AdapterLinear")
