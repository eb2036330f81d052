"""Products with 4-bit weights on rows up to the largest float: finite where the product is,
on both sides of the rows that read the packed weight, beside rows of any other size."""
import pytest
import torch

import experts_reference as xr
import ops_reference as ref
from test_gpu_quant4 import _cuda, _pack

pytestmark = pytest.mark.gpu


def _weights(n, N, K, group, zeros, seed):
    """Scales of about 2^-14: the largest row's outputs stay below 2^127 whatever its signs."""
    g = torch.Generator().manual_seed(seed)
    groups = -(-K // group)
    q = torch.randint(0, 16, (n, N, K), generator=g, dtype=torch.uint8)
    scale = (torch.rand(n, N, groups, generator=g) + 0.25) * 2.0 ** -14
    zero = torch.randint(0, 16, (n, N, groups), generator=g, dtype=torch.uint8) if zeros else None
    return q, scale, zero


def _rows(dtype, P, K, signs, seed):
    """Rows of sizes from 2^-100 up, of each kind in every tile, the largest float among them."""
    g = torch.Generator().manual_seed(seed)
    most = float(torch.finfo(xr.DT[dtype]).max)
    p = torch.tensor([127, -100, 118, 0, 120, 117, 40, 124])[torch.arange(P) % 8].double()
    x = (1 + torch.rand(P, K, generator=g).double()) * 2 ** p.unsqueeze(1)
    if signs == "mixed":
        x = torch.where(torch.rand(P, K, generator=g) < 0.5, -x, x)
    elif signs == "negative":
        x = -x
    x[::8, ::3] = torch.where(x[::8, ::3] > 0, most, -most)
    return x.clamp(-most, most).to(xr.DT[dtype])


def _check(dtype, P, N, K, group, zeros, signs, gate=None, n=1, bank=False):
    from fp32_emulated_gemm_amd.experts import experts_lib, sort_tokens
    from fp32_emulated_gemm_amd.quant4 import quant4_linear
    q, scale, zero = _weights(n, N, K, group, zeros, P + K)
    if gate is not None:
        scale[:, :N // 2] = 0                              # gates of 0: half of the up projection
    x = _rows(dtype, P, K, signs, P)
    order, offsets = None, torch.tensor([0, P])
    if bank:
        ids = (torch.arange(P) * n // P).int().unsqueeze(1)
        offsets, order = xr.order(ids, n)[0], sort_tokens(ids.cuda(), n)
    few = experts_lib().sgemm_emu_quant4_linear_workspace(0 if dtype == "f32" else 1, P, N, K, n, group, zeros) == 0
    y = quant4_linear(x.cuda(), _pack(q, scale, _cuda(zero), group, bank), None, gate, order)
    assert bool(y.isfinite().all())
    h, bound = xr.quant4(x, q, scale, zero, group, offsets, None, gate, few)
    assert float(h.abs().max()) < 2.0 ** 127
    # the second sums of a row that passed the range are multiples of 2^-149 2^12
    ref.check(y, (h, bound - ref.TINY + K * 2.0 ** -137), "y")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("P,N,K", [(1, 16, 128), (1, 130, 384), (7, 34, 500), (16, 64, 512), (40, 48, 256), (64, 96, 130),
                                   (65, 96, 130), (129, 48, 256)])
@pytest.mark.parametrize("signs,zeros", [("positive", True), ("negative", False), ("mixed", True)])
def test_rows_up_to_the_largest_float(dtype, group, P, N, K, signs, zeros):
    _check(dtype, P, N, K, group, zeros, signs)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("signs", ["positive", "mixed"])
@pytest.mark.parametrize("P,n", [(3, 1), (16, 2), (60, 2), (64, 1)])
def test_with_a_gate_and_experts(dtype, signs, P, n):
    _check(dtype, P, 96, 256, 128, True, signs, "sigmoid")
    _check(dtype, P, 40, 256, 64, False, signs, None, n, True)
    _check(dtype, P, 96, 300, 32, True, signs, "sigmoid", n, True)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("P", [1, 8, 33])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_infinities_stay_in_their_rows(dtype, P, bad):
    """A row with one is NaN; rows beside it, large ones too, keep their values."""
    from fp32_emulated_gemm_amd.quant4 import quant4_linear
    q, scale, zero = _weights(1, 48, 256, 64, True, 5)
    x = _rows(dtype, P, 256, "positive", 5)
    w4 = _pack(q, scale, zero, 64, False)
    want = quant4_linear(x.cuda(), w4)
    x[P // 2, 17] = bad
    got = quant4_linear(x.cuda(), w4)
    assert bool(got[P // 2].isnan().all())
    rest = torch.arange(P, device="cuda") != P // 2
    assert bool(want.isfinite().all()) and torch.equal(got[rest], want[rest])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("group", [32, 128])
@pytest.mark.parametrize("P", [1, 8, 40])
def test_the_last_expert_of_a_bank_past_32_bits(dtype, group, P):
    """Values, scales and zeros of more than 2^32 bytes of packed weights, at the derived bounds."""
    from fp32_emulated_gemm_amd.experts import sort_tokens
    from fp32_emulated_gemm_amd.quant4 import pack, quant4_linear
    n, N, K, rows = 72, 10240, 12288, 16
    q, scale, zero = _weights(1, rows, K, group, True, P)
    full = torch.zeros(n, N, K, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(n, N, K // group, device="cuda")
    zeros = torch.zeros(n, N, K // group, dtype=torch.uint8, device="cuda")
    full[-1, -rows:], scales[-1, -rows:], zeros[-1, -rows:] = q[0].cuda(), scale[0].cuda(), zero[0].cuda()
    w4 = pack(full, scales, zeros, group)
    assert w4.packed.numel() > 1 << 32
    del full, scales, zeros
    x = torch.randn(P, K, generator=torch.Generator().manual_seed(P)).to(xr.DT[dtype])
    y = quant4_linear(x.cuda(), w4, order=sort_tokens(torch.full((P,), n - 1, dtype=torch.int32, device="cuda"), n))
    assert not bool(y[:, :-rows].any())
    ref.check(y[:, -rows:], xr.quant4(x, q, scale, zero, group, torch.tensor([0, P]), None, None, True), "y")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("symmetric", [True, False])
def test_the_largest_weights_stay_finite(dtype, symmetric):
    """Groups up to the largest float stand for finite weights, in both types, a step off at most."""
    from fp32_emulated_gemm_amd.quant4 import pack, quantize_values
    most = float(torch.finfo(xr.DT[dtype]).max)
    w = torch.randn(6, 256, generator=torch.Generator().manual_seed(1)).double()
    w = w / w.abs().amax(1, keepdim=True) * most
    w[0], w[1, ::2], w[1, 1::2] = most, most, -most
    w[2], w[3] = -most, w[3].abs()
    w[4, :] = torch.where(torch.arange(256) % 32 == 0, -most / 64, most)
    w = w.clamp(-most, most).to(xr.DT[dtype])
    q, scale, zero = quantize_values(w.cuda(), 32, symmetric)
    w4 = pack(q, scale, zero, 32)
    assert bool(scale.isfinite().all())
    for out in (torch.float32, torch.bfloat16):
        got = w4.dequantize(out)
        assert bool(got.isfinite().all())
        # half a step, another half where the zero point is rounded, and what the limited scale s leaves out:
        # the levels end at m s = B, the largest bfloat16, m = max(z, 15 - z) from 8 to 15, the weights at
        # B (1 + 2^-8), m 2^-8 s further; the scale without the limit is at most z (1 + 2^-8) / (z - 1/2) s,
        # so that the other end lies at most 7.5 8 / 7.5 (1 + 2^-8) - 7 < 1 + 15 2^-8 steps off (z = 8).
        # In bfloat16 the weight's own rounding comes to it.
        step = scale.double().repeat_interleave(32, 1).cpu()
        room = step * ((0.5 if symmetric else 1.0) + 15 * 2.0 ** -8) + (2.0 ** -8 * got.double().cpu().abs() if out is torch.bfloat16 else 0)
        assert bool(((got.double().cpu() - w.double()).abs() <= room).all())
