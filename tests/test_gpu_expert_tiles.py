"""The experts' products at sizes that take every tile and both parts of a launch of
256 x 256 tiles, against float64 on the GPU."""
import pytest
import torch

import experts_reference as xr
import ops_reference as ref

pytestmark = pytest.mark.gpu


def _run(dtype, counts, spare, N, K, gate, seed=0):
    """Rows given directly: counts[e] of each expert, then `spare` of none."""
    from fp32_emulated_gemm_amd.experts import ExpertOrder, expert_linear
    g = torch.Generator("cuda").manual_seed(seed)
    n, used = len(counts), sum(counts)
    P = used + spare
    offsets = [0]
    for c in counts:
        offsets.append(offsets[-1] + c)
    places = torch.arange(P, dtype=torch.int32).view(P, 1)
    order = ExpertOrder(torch.tensor(offsets, dtype=torch.int32).cuda(), places.view(-1).cuda(), places.cuda(), n)

    def normal(*shape, sigma=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * sigma).to(xr.DT[dtype])

    x, w, dh = normal(P, K), normal(n, N, K, sigma=K ** -0.5), normal(P, N // 2 if gate else N)
    x[used:], dh[used:] = float("nan"), float("nan")
    x.requires_grad_(True), w.requires_grad_(True)
    h = expert_linear(x, w, order, gate=gate)
    dx, dw = torch.autograd.grad(h, (x, w), dh)
    return x.detach(), w.detach(), dh, offsets, h.detach(), dx, dw


def _compare(dtype, counts, spare, N, K, gate):
    """Every element within the bounds of experts_reference, computed on the GPU in float64."""
    x, w, dh, offsets, h, dx, dw = _run(dtype, counts, spare, N, K, gate)
    used = offsets[-1]
    want = xr.experts(x[:used], w, torch.tensor(offsets), None, gate, dh[:used])
    for got, name in ((h, "h"), (dx, "dx")):
        assert bool((got[used:] == 0).all()), name
        ref.check(got[:used], tuple(t.cpu() for t in want[name]), name)
    ref.check(dw, tuple(t.cpu() for t in want["dw"]), "dw")


@pytest.mark.parametrize("counts,spare,N,K,gate", [
    ([700, 0, 1300, 250], 30, 1024, 512, None),          # few tiles
    ([2100, 1800, 900, 3000, 1], 200, 2048, 256, "silu"),
    ([5000, 2600, 4100], 0, 1400, 640, "gelu"),          # an F that is no multiple of 16
    ([6000], 10, 2304, 448, None),
    ([4000, 257, 4300, 8000], 5, 2048, 512, "silu"),     # whole rounds and a rest
    ([130] * 40, 3, 776, 136, None)])
def test_bfloat16_tiles(counts, spare, N, K, gate):
    _compare("bf16", counts, spare, N, K, gate)


@pytest.mark.parametrize("counts,spare,N,K,gate", [
    ([700, 0, 1300, 250], 30, 1024, 256, "gelu"), ([2100, 1800, 900], 20, 1030, 131, None), ([4000], 0, 512, 512, None),
    # weights of whole allocations, whose ends the steps loaded ahead must not pass
    ([512], 0, 2048, 2048, None), ([128], 0, 1024, 1024, None)])
def test_float32_tiles(counts, spare, N, K, gate):
    _compare("f32", counts, spare, N, K, gate)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_results_repeat(dtype):
    """Bit for bit, the gradients too."""
    first, second = (_run(dtype, [900, 0, 2500, 300], 12, 1536, 384, "silu")[4:] for _ in range(2))
    for a, b in zip(first, second):
        assert torch.equal(a, b)
