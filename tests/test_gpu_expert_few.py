"""The experts' products of few rows, on both sides of the sizes where other kernels take
them, against the 64-bit definition at derived bounds."""
import pytest
import torch

import experts_reference as xr
import ops_reference as ref
from test_gpu_experts import _check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,k,n,N,K", [
    (1, 1, 1, 2, 3), (1, 1, 1, 34, 127), (1, 3, 7, 30, 129), (2, 1, 1, 16, 1024), (7, 2, 5, 18, 2050), (15, 1, 1, 64, 128),
    (16, 1, 2, 96, 250), (17, 1, 1, 98, 385), (64, 4, 3, 62, 136), (256, 1, 1, 128, 72), (257, 1, 1, 128, 72),
    (128, 2, 40, 66, 1025), (129, 2, 40, 66, 1025), (3, 2, 1024, 32, 64),
    (1000, 1, 1, 34, 333), (512, 2, 3, 48, 700), (1025, 1, 2, 34, 333)])
@pytest.mark.parametrize("gate,bias", [(None, True), ("silu", True), ("relu", False)])
def test_few_rows(dtype, T, k, n, N, K, gate, bias):
    _check(dtype, T, k, n, N, K, gate, bias, "mixed", seed=T + N)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["one", "none", "few", "full"])
@pytest.mark.parametrize("K", [64, 333])
def test_experts_without_rows(dtype, kind, K):
    _check(dtype, 31, 3, 6, 80, K, "gelu", True, kind)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("K,ld,at", [(130, 132, 0), (130, 132, 2), (129, 140, 1), (128, 129, 0), (31, 32, 0), (255, 256, 0)])
def test_strided_rows(dtype, K, ld, at):
    """What lies beside the rows is not read into them: NaN there."""
    from fp32_emulated_gemm_amd.experts import expert_linear, sort_tokens
    P, N, n = 19, 40, 2
    g = torch.Generator().manual_seed(K + ld)
    wide = torch.full((P, ld + at), float("nan"), dtype=xr.DT[dtype])
    wide[:, at:at + K] = torch.randn(P, K, generator=g).to(wide.dtype)
    w = (torch.randn(n, N, K, generator=g) * K ** -0.5).to(wide.dtype)
    ids = (torch.arange(P) % n).int().unsqueeze(1)
    offsets = xr.order(ids, n)[0]
    x = wide[:, at:at + K]
    got = expert_linear(wide.cuda()[:, at:at + K], w.cuda(), sort_tokens(ids.cuda(), n))
    ref.check(got, xr.experts(x, w, offsets, None, None, torch.zeros(P, N).to(w.dtype))["h"], "h")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_captured_and_repeated(dtype):
    """A single token's layer from a graph, bit for bit as called, with other rows in each replay."""
    from fp32_emulated_gemm_amd.experts import ExpertFeedForward
    torch.manual_seed(0)
    m = ExpertFeedForward(200, 136, 9, bias=True, device="cuda", dtype=xr.DT[dtype])
    x, ids = torch.randn(1, 200, device="cuda").to(xr.DT[dtype]), torch.tensor([[3, 8]], dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.no_grad():
        m(x, ids)
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            y = m(x, ids)
        for i in range(4):
            x.copy_(torch.randn(1, 200, device="cuda"))
            ids.copy_(torch.tensor([[i, 8 - 2 * i]], dtype=torch.int32))
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(y, m(x, ids))
