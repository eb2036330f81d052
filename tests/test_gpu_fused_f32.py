"""The float32 products with the gate or the adapters' part in them, on grids of more
128 x 128 tiles than the GPU has CUs: the kernel that copies both operands' planes
(1024 rows and 4096 columns or more), and workgroups that go on to a second tile,
restarting their accumulators and reloading the bias while copies are under way."""
import pytest
import torch

import ops_reference as ref
from test_gpu_adapters import _check as check_adapter, _ids, _inputs as adapter_inputs, _run as run_adapter
from test_gpu_gated import _inputs as gated_inputs, _run as run_gated

pytestmark = pytest.mark.gpu

TILE = 128


def _more_tiles_than_cus(M, N, K):
    """One pass over K per 128 x 128 tile: no stream-K, and too many tiles for 64 x 64 ones."""
    import fp32_emulated_gemm_amd as fe
    assert fe.sgemm_emu_split_k(M, N, K) == 1
    tiles = -(-M // TILE) * -(-N // TILE)
    assert tiles > torch.cuda.get_device_properties(0).multi_processor_count


# outputs F (N = 2 F columns), planes of A or A split in the kernel; the last adds K's padding
GATED = [(1100, 128, 2100), (1300, 192, 2049), (6200, 256, 1024), (4200, 320, 700), (1100, 100, 2100), (6200, 250, 1024)]


@pytest.mark.parametrize("M,K,F", GATED)
def test_gated(M, K, F):
    _more_tiles_than_cus(M, 2 * F, K)
    x, w, b, dh = gated_inputs("f32", M, K, F, True, seed=M)
    want = ref.gated(x, w, b, "gelu", dh)
    got = run_gated(x, w, b, dh, "gelu")
    for name in ("h0", "h", "dx", "dw", "db"):
        ref.check(got[name], want[name.rstrip("0")], name)
    assert torch.equal(got["h0"], got["h"])


@pytest.mark.parametrize("gate", ["silu", "gelu_tanh", "sigmoid"])
@pytest.mark.parametrize("M,K,F", GATED[:3:2])
def test_gates(M, K, F, gate):
    from fp32_emulated_gemm_amd.gated import gated_linear, plan_weight
    x, w, b, _ = gated_inputs("f32", M, K, F, True, seed=K)
    xs, ws, bs = x.cuda(), w.cuda(), b.cuda()
    first = gated_linear(xs, ws, bs, gate=gate, plan=plan_weight(ws))
    ref.check(first, ref.gated(x, w, b, gate)["h"], gate)
    for _ in range(3):
        assert torch.equal(gated_linear(xs, ws, bs, gate=gate), first)


@pytest.mark.parametrize("kind", ["spans", "mixed"])
@pytest.mark.parametrize("M,K,N,n,r", [(1100, 128, 4200, 5, 8), (1300, 192, 4100, 3, 13), (6200, 256, 1024, 7, 16),
                                       (4200, 320, 1400, 4, 5), (4200, 100, 1400, 4, 8), (1100, 131, 4200, 3, 4)])
def test_adapters(M, K, N, n, r, kind):
    _more_tiles_than_cus(M, N, K)
    t = adapter_inputs("f32", M, K, N, n, r, seed=M)
    ids = _ids(kind, M, n)
    got = run_adapter(t, ids)
    check_adapter(t, ids, got, f"{M}x{K}x{N}")
    again = run_adapter(t, ids, plan=True)
    for name in got:
        assert torch.equal(got[name], again[name]), name
