"""Weights of 4 bits: quantised, packed and unpacked bit for bit, and their products
against the 64-bit definition at derived bounds."""
import pytest
import torch

import experts_reference as xr
import ops_reference as ref

pytestmark = pytest.mark.gpu


def _weights(n, N, K, group, zeros, seed=0):
    g = torch.Generator().manual_seed(seed)
    groups = -(-K // group)
    q = torch.randint(0, 16, (n, N, K), generator=g, dtype=torch.uint8)
    scale = (torch.rand(n, N, groups, generator=g) + 0.25) * 0.3 * max(K, 1) ** -0.5
    scale = torch.where(torch.rand(n, N, groups, generator=g) < 0.1, -scale, scale)
    zero = torch.randint(0, 16, (n, N, groups), generator=g, dtype=torch.uint8) if zeros else None
    return q, scale, zero


def _cuda(t):
    return None if t is None else t.cuda()


def _pack(q, scale, zero, group, bank):
    from fp32_emulated_gemm_amd.quant4 import pack
    if not bank:
        q, scale, zero = q[0], scale[0], None if zero is None else zero[0]
    return pack(q.cuda(), scale.cuda(), _cuda(zero), group)


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("n,N,K", [(1, 1, 1), (1, 16, 128), (3, 17, 129), (2, 40, 300), (5, 33, 64), (1, 0, 5), (1, 5, 0)])
@pytest.mark.parametrize("zeros", [True, False])
def test_packed_and_back(group, n, N, K, zeros):
    q, scale, zero = _weights(n, N, K, group, zeros)
    w4 = _pack(q, scale, zero, group, True)
    column = torch.arange(K) // group
    z = 8.0 if zero is None else zero.float()[..., column]
    want = (q.float() - z) * scale[..., column]          # one rounding, as the kernel's
    assert torch.equal(w4.dequantize().cpu(), want)
    assert torch.equal(w4.dequantize(torch.bfloat16).cpu(), want.bfloat16())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("group", [32, 128])
@pytest.mark.parametrize("symmetric", [True, False])
@pytest.mark.parametrize("shape", [(3, 50), (2, 17, 300), (4, 128)])
def test_quantized_to_nearest(dtype, group, symmetric, shape):
    from fp32_emulated_gemm_amd.quant4 import quantize, quantize_values
    g = torch.Generator().manual_seed(1)
    w = torch.randn(shape, generator=g).to(xr.DT[dtype])
    w[..., 0, :] = 0.0                                    # groups of zeros
    w[..., 1, :] = w[..., 1, :].abs() + 0.5               # one sign
    q, scale, zero = quantize_values(w.cuda(), group, symmetric)
    w4 = quantize(w.cuda(), group, symmetric).dequantize().cpu().double()
    column = torch.arange(shape[-1]) // group
    s = scale.cpu().double()[..., column]
    pad = -shape[-1] % group
    parts = torch.nn.functional.pad(w.double(), (0, pad)).unflatten(-1, (-1, group))
    if symmetric:
        assert zero is None
        want = parts.abs().amax(-1) / 7
    else:
        want = (parts.amax(-1).clamp(min=0) - parts.amin(-1).clamp(max=0)) / 15
        assert int(zero.max()) <= 15
    # two roundings of 2^-24 in the quotients by constants, one in the difference
    assert ((scale.cpu().double() - want).abs() <= 4 * ref.U * want.abs() * 2).all()
    assert int(q.max()) <= 15
    # nearest: half a step, and with a rounded zero point another half at the ends of the range
    assert ((w4 - w.double()).abs() <= s * (0.5 if symmetric else 1.0) * (1 + 2.0 ** -18)).all()
    assert (w4[..., 0, :] == 0).all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("symmetric", [True, False])
def test_groups_that_are_not_finite_stand_for_nan(bad, symmetric):
    from fp32_emulated_gemm_amd.quant4 import quantize
    w = torch.randn(3, 100, device="cuda")
    w[1, 40] = bad
    got = quantize(w, 32, symmetric).dequantize()
    assert got[1, 32:64].isnan().all()
    got[1, 32:64] = 0.0
    assert got.isfinite().all()


def _products(dtype, T, k, n, N, K, group, zeros, gate, bias, kind="mixed", seed=0):
    """k = 0: a layer."""
    from fp32_emulated_gemm_amd.experts import sort_tokens
    from fp32_emulated_gemm_amd.experts import experts_lib
    from fp32_emulated_gemm_amd.quant4 import quant4_linear
    g = torch.Generator().manual_seed(seed)
    P = T * max(k, 1)
    x = torch.randn(P, K, generator=g).to(xr.DT[dtype])
    b = (torch.randn(n, N, generator=g) * 0.1).to(x.dtype) if bias else None
    q, scale, zero = _weights(n, N, K, group, zeros, seed)
    w4 = _pack(q, scale, zero, group, k > 0)
    order, offsets = None, torch.tensor([0, P])
    if k > 0:
        ids = xr.make_ids(kind, T, k, n, seed)
        offsets = xr.order(ids, n)[0]
        order = sort_tokens(ids.cuda(), n)
        x[offsets[-1]:] = float("nan")
    code = 0 if dtype == "f32" else 1
    few = experts_lib().sgemm_emu_quant4_linear_workspace(code, P, N, K, n, group, zeros) == 0
    bd = None if b is None else b.cuda() if k > 0 else b[0].cuda()
    y = quant4_linear(x.cuda(), w4, bd, gate, order)
    return ref.check(y, xr.quant4(x, q, scale, zero, group, offsets, b, gate, few), "y"), few


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("T,N,K", [(1, 2, 1), (1, 64, 128), (1, 130, 1000), (3, 34, 129), (16, 96, 256), (17, 66, 500),
                                   (33, 48, 64), (64, 320, 384), (65, 96, 160), (128, 48, 200),
                                   (129, 64, 96), (300, 130, 257)])
@pytest.mark.parametrize("gate,bias,zeros", [(None, True, True), ("silu", False, True), ("gelu", True, False)])
def test_layers(dtype, group, T, N, K, gate, bias, zeros):
    _products(dtype, T, 0, 1, N, K, group, zeros, gate, bias, seed=T + K)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("group", [32, 128])
@pytest.mark.parametrize("T,k,n,N,K", [(1, 2, 8, 64, 200), (16, 2, 32, 40, 128), (40, 3, 5, 34, 300), (30, 2, 2, 96, 64),
                                       (100, 2, 3, 66, 130)])
@pytest.mark.parametrize("kind", ["mixed", "one", "none", "few"])
@pytest.mark.parametrize("gate", [None, "silu"])
def test_experts(dtype, group, T, k, n, N, K, kind, gate):
    _products(dtype, T, k, n, N, K, group, True, gate, True, kind, seed=T)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,k,n,N,K", [(0, 0, 1, 8, 8), (3, 0, 1, 0, 8), (3, 0, 1, 8, 0), (100, 0, 1, 8, 0), (4, 0, 1, 6, 4),
                                       (4, 2, 0, 8, 8), (0, 2, 3, 8, 8)])
@pytest.mark.parametrize("gate", [None, "relu"])
def test_empty(dtype, T, k, n, N, K, gate):
    _products(dtype, T, k, n, N, K, 64, True, gate, True, "none" if n == 0 else "mixed")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_ends_of_the_range(dtype):
    """float32 keeps its relative precision for the smallest and largest rows: the parts are scaled."""
    from fp32_emulated_gemm_amd.quant4 import quant4_linear
    g = torch.Generator().manual_seed(3)
    q, scale, zero = _weights(1, 32, 256, 64, True)
    x = torch.randn(8, 256, generator=g) * torch.tensor([2.0 ** p for p in (-120, -100, -60, 0, 30, 60, 90, 110)]).unsqueeze(1)
    x = x.to(xr.DT[dtype])
    scale = scale.abs() * 2.0 ** torch.randint(-6, 6, scale.shape, generator=g)
    y = quant4_linear(x.cuda(), _pack(q, scale, zero, 64, False))
    h, bound = xr.quant4(x, q, scale, zero, 64, torch.tensor([0, 8]), None, None, True)
    ref.check(y, (h, bound - ref.TINY + 2.0 ** -140), "y")
