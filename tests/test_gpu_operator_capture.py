"""Float32 calls whose products take stream-K, on a stream being captured into a graph:
refused with nothing recorded, whatever the call does before its products."""
import pytest
import torch

pytestmark = pytest.mark.gpu

F32 = 0
MARK = 3.0


def _gated(L, keep):
    M, F, K = 129, 65, 1024
    x, w, b = torch.randn(M, K), torch.randn(2 * F, K) * K ** -0.5, torch.randn(2 * F)
    t = {k: v.cuda() for k, v in (("x", x), ("w", w), ("b", b))}
    out = {"h": torch.empty(M, F, device="cuda")}
    if keep:
        out["z"] = torch.empty(M, 2 * 72, device="cuda")
    zp = out["z"].data_ptr() if keep else None
    n = L.sgemm_emu_gated_linear_workspace(F32, M, F, K, t["x"].data_ptr(), K, t["w"].data_ptr(), K, None, zp)
    out["ws"] = torch.empty(n // 4, device="cuda")

    def call(stream):
        return L.sgemm_emu_gated_linear(F32, M, F, K, t["x"].data_ptr(), K, t["w"].data_ptr(), K, None,
                                        t["b"].data_ptr(), 0, out["h"].data_ptr(), F, zp, out["ws"].data_ptr(), n, stream)
    return [(M, 2 * F, K, True)], call, out, t


def _gated_backward(L, _):
    M, F, K = 1024, 65, 130               # dW's product takes stream-K, dX's before it does not
    pitch = 2 * 72
    t = {"x": torch.randn(M, K).cuda(), "w": torch.randn(2 * F, K).cuda(), "z": torch.randn(M, pitch).cuda(),
         "dh": torch.randn(M, F).cuda()}
    out = {"dx": torch.empty(M, K, device="cuda"), "dw": torch.empty(2 * F, K, device="cuda"),
           "db": torch.empty(2 * F, device="cuda")}
    n = L.sgemm_emu_gated_linear_backward_workspace(F32, M, F, K)
    out["ws"] = torch.empty(n // 4, device="cuda")

    def call(stream):
        return L.sgemm_emu_gated_linear_backward(
            F32, M, F, K, t["x"].data_ptr(), K, t["w"].data_ptr(), K, t["z"].data_ptr(), 0, t["dh"].data_ptr(), F,
            out["dx"].data_ptr(), K, out["dw"].data_ptr(), K, out["db"].data_ptr(), out["ws"].data_ptr(), n, stream)
    return [(M, K, 2 * 96, False), (2 * F, K, M, True)], call, out, t


def _adapter_inputs(M, N, K, n, r):
    return {"x": torch.randn(M, K).cuda(), "w": torch.randn(N, K).cuda(), "a": torch.randn(n, r, K).cuda(),
            "b": torch.randn(n, N, r).cuda(), "ids": (torch.arange(M) % n).int().cuda(), "dy": torch.randn(M, N).cuda()}


def _adapter(L, keep):
    M, N, K, n, r = 129, 130, 1024, 3, 4
    t = _adapter_inputs(M, N, K, n, r)
    p = {k: v.data_ptr() for k, v in t.items()}
    out = {"y": torch.empty(M, N, device="cuda")}
    if keep:
        out["s"] = torch.empty(M, 16, device="cuda")
    sp = out["s"].data_ptr() if keep else None
    nws = L.sgemm_emu_adapter_linear_workspace(F32, M, N, K, p["x"], K, p["w"], K, None, n, r, p["b"], sp)
    out["ws"] = torch.empty(nws // 4, device="cuda")

    def call(stream):
        return L.sgemm_emu_adapter_linear(F32, M, N, K, p["x"], K, p["w"], K, None, None, n, r, p["a"], p["b"], None,
                                          p["ids"], out["y"].data_ptr(), N, sp, out["ws"].data_ptr(), nws, stream)
    return [(M, N, K, True)], call, out, t


def _adapter_backward(L, _):
    M, N, K, n, r = 129, 1024, 130, 3, 4
    t = _adapter_inputs(M, N, K, n, r)
    t["s"] = torch.randn(M, 16).cuda()
    size = L.sgemm_emu_plan_bytes(F32, N, K, 1)
    t["plan"] = torch.empty(size // 4, device="cuda")
    p = {k: v.data_ptr() for k, v in t.items()}
    assert L.sgemm_emu_plan_weight(F32, N, K, p["w"], K, 1, p["plan"], torch.cuda.current_stream().cuda_stream) == 0
    out = {"dx": torch.empty(M, K, device="cuda"), "da": torch.empty(n, r, K, device="cuda"),
           "db": torch.empty(n, N, r, device="cuda")}
    nws = L.sgemm_emu_adapter_linear_backward_workspace(F32, M, N, K, n, r)
    out["ws"] = torch.empty(nws // 4, device="cuda")

    def call(stream):
        return L.sgemm_emu_adapter_linear_backward(
            F32, M, N, K, p["x"], K, p["plan"], n, r, p["a"], p["b"], None, p["ids"], p["s"], p["dy"], N,
            out["dx"].data_ptr(), K, out["da"].data_ptr(), out["db"].data_ptr(), out["ws"].data_ptr(), nws, stream)
    return [(M, K, N, True)], call, out, t


@pytest.mark.parametrize("make", [_gated, _gated_backward, _adapter, _adapter_backward])
@pytest.mark.parametrize("keep", [False, True])
def test_refused_captures_record_nothing(make, keep):
    """Outputs and workspace keep their marks through replays of the graph; the same call then runs
    eagerly, before and after giving the same bits."""
    import fp32_emulated_gemm_amd as fe
    from fp32_emulated_gemm_amd.ops import ops_lib
    torch.manual_seed(7)
    products, call, out, held = make(ops_lib(), keep)
    for M, N, K, streamk in products:
        assert (fe.sgemm_emu_split_k(M, N, K) > 1) == streamk
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    assert call(stream.cuda_stream) == fe.SGEMM_EMU_OK
    stream.synchronize()
    first = {k: v.clone() for k, v in out.items() if k != "ws"}
    counter = torch.zeros(1, device="cuda")
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        counter.add_(1)
        status = call(stream.cuda_stream)
    assert status == fe.SGEMM_EMU_ECAPTURE
    for k in range(3):
        for v in out.values():
            v.fill_(MARK)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert counter.item() == k + 1
        for name, v in out.items():
            assert bool((v == MARK).all()), f"the refused call recorded work on {name}"
        assert call(stream.cuda_stream) == fe.SGEMM_EMU_OK
        stream.synchronize()
        for name, v in first.items():
            if name != "z":                   # whose padding columns are not set
                assert torch.equal(out[name], v), name
    del graph, held
