"""Checks of the operators' C ABI (include/sgemm_emu_ops.h) that need no GPU: every
function declared, exported and bound, the header's C99 and C++17, the sizes of
plans, arguments refused before any HIP call, and the tensor functions' refusals."""
import ctypes
import os
import re
import shutil
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "sgemm_emu_ops.h")
P = 0x10000  # any nonzero, 256-byte aligned address: never dereferenced on these paths
F32, BF16 = 0, 1
EINVAL, ENULL, EARCH = -1, -2, -3


def _declared():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    return sorted(set(re.findall(r"^(?:int|int64_t)\s+(\w+)\s*\(", text, flags=re.M)))


@pytest.fixture(scope="module")
def L():
    from fp32_emulated_gemm_amd import ops
    return ops.ops_lib()


def test_declared_exported_and_bound(L):
    import fp32_emulated_gemm_amd as fe
    from fp32_emulated_gemm_amd import ops
    assert _declared() == sorted(ops.OPS_EXPORTS)
    libs = [L]
    if not os.environ.get("SGEMM_EMU_LIB_OVERRIDE"):
        libs.append(ctypes.CDLL(os.path.join(os.path.dirname(os.path.abspath(fe.__file__)),
                                             "libsgemm_emu_serial_lds.so")))
    for lib in libs:
        for name in _declared():
            assert hasattr(lib, name), name


def test_header_in_c_and_cxx(tmp_path):
    if shutil.which("gcc") is None or shutil.which("g++") is None:
        pytest.skip("no host C compiler")
    src = tmp_path / "ops.c"
    src.write_text('#include "sgemm_emu_ops.h"\nint main(void) { return (int)SGEMM_EMU_F32; }\n')
    inc = os.path.join(ROOT, "include")
    for cc in (["gcc", "-std=c99", "-pedantic"], ["g++", "-std=c++17", "-x", "c++"]):
        subprocess.run([*cc, "-Wall", "-Wextra", "-Werror", "-I", inc, "-c", str(src), "-o", str(tmp_path / "o")],
                       check=True)


def test_plan_bytes(L):
    pad = lambda k: (k + 63) // 64 * 64   # noqa: E731
    for rows, cols in ((0, 5), (5, 0), (1, 1), (10, 64), (10, 65), (130, 1000)):
        assert L.sgemm_emu_plan_bytes(F32, rows, cols, 0) == 6 * rows * pad(cols)
        assert L.sgemm_emu_plan_bytes(BF16, rows, cols, 0) == 2 * rows * pad(cols)
        assert L.sgemm_emu_plan_bytes(F32, rows, cols, 1) == 6 * cols * pad(rows)
    assert L.sgemm_emu_plan_bytes(F32, 6, 65, 2) == 6 * 6 * 128
    for bad in ((2, 4, 4, 0), (F32, -1, 4, 0), (F32, 4, 1 << 40, 0), (F32, 4, 4, 3), (F32, 5, 4, 2)):
        assert L.sgemm_emu_plan_bytes(*bad) == EINVAL
    assert L.sgemm_emu_plan_weight(F32, 4, 4, 0, 4, 0, P, None) == ENULL
    assert L.sgemm_emu_plan_weight(F32, 4, 4, P, 4, 0, 0, None) == ENULL
    assert L.sgemm_emu_plan_weight(F32, 4, 4, P, 3, 0, P, None) == EINVAL
    assert L.sgemm_emu_plan_weight(F32, 4, 4, P + 2, 4, 0, P, None) == EINVAL
    assert L.sgemm_emu_plan_weight(F32, 4, 4, P, 4, 0, P + 8, None) == EINVAL
    assert L.sgemm_emu_plan_weight(F32, 0, 4, 0, 4, 0, 0, None) == 0


def _gated(L, dt=F32, M=4, F=4, K=8, X=P, ldx=8, W=P, ldw=8, plan=0, bias=0, gate=0, H=P, ldh=4, Z=0):
    return L.sgemm_emu_gated_linear(dt, M, F, K, X, ldx, W, ldw, plan, bias, gate, H, ldh, Z, None, 0, None)


@pytest.mark.parametrize("bad,status", [
    (dict(dt=2), EINVAL), (dict(M=-1), EINVAL), (dict(F=-1), EINVAL), (dict(K=-1), EINVAL), (dict(F=1 << 22), EINVAL),
    (dict(gate=5), EINVAL), (dict(gate=-1), EINVAL), (dict(ldx=7), EINVAL), (dict(ldw=7), EINVAL),
    (dict(ldh=3), EINVAL), (dict(ldx=1 << 24), EINVAL), (dict(X=0), ENULL), (dict(W=0), ENULL), (dict(H=0), ENULL),
    (dict(X=P + 2), EINVAL), (dict(dt=BF16, X=P + 1), EINVAL), (dict(bias=P + 2), EINVAL), (dict(plan=P + 8), EINVAL),
    (dict(Z=P + 8), EINVAL), (dict(M=0, X=0, H=0), 0), (dict(F=0, W=0, H=0), 0)], ids=str)
def test_gated_arguments(L, bad, status):
    assert _gated(L, **bad) == status


def _gated_back(L, dt=F32, M=4, F=4, K=8, X=P, ldx=8, W=P, ldw=8, Z=P, gate=0, dH=P, lddh=4, dX=P, lddx=8, dW=P,
                lddw=8, db=P):
    return L.sgemm_emu_gated_linear_backward(dt, M, F, K, X, ldx, W, ldw, Z, gate, dH, lddh, dX, lddx, dW, lddw, db,
                                             None, 0, None)


@pytest.mark.parametrize("bad,status", [
    (dict(dt=-1), EINVAL), (dict(gate=9), EINVAL), (dict(Z=0), ENULL), (dict(Z=P + 4), EINVAL), (dict(dH=0), ENULL),
    (dict(X=0), ENULL), (dict(W=0), ENULL), (dict(lddx=7), EINVAL), (dict(lddw=7), EINVAL), (dict(lddh=3), EINVAL),
    (dict(db=P + 2), EINVAL)], ids=str)
def test_gated_backward_arguments(L, bad, status):
    assert _gated_back(L, **bad) == status


def _adapter(L, dt=F32, M=4, N=4, K=8, X=P, ldx=8, W=P, ldw=8, plan=0, bias=0, n=2, r=2, down=P, up=P, scale=0, ids=P,
             Y=P, ldy=4, S=0):
    return L.sgemm_emu_adapter_linear(dt, M, N, K, X, ldx, W, ldw, plan, bias, n, r, down, up, scale, ids, Y, ldy, S,
                                      None, 0, None)


@pytest.mark.parametrize("bad,status", [
    (dict(dt=2), EINVAL), (dict(M=-1), EINVAL), (dict(n=-1), EINVAL), (dict(r=-1), EINVAL), (dict(n=65536), EINVAL),
    (dict(ldx=7), EINVAL), (dict(ldw=7), EINVAL), (dict(ldy=3), EINVAL), (dict(X=0), ENULL), (dict(W=0), ENULL),
    (dict(Y=0), ENULL), (dict(down=0), ENULL), (dict(up=0), ENULL), (dict(ids=0), ENULL), (dict(ids=P + 2), EINVAL),
    (dict(scale=P + 1), EINVAL), (dict(bias=P + 1), EINVAL), (dict(S=P + 4), EINVAL), (dict(plan=P + 4), EINVAL),
    (dict(M=0, X=0, Y=0, ids=0), 0), (dict(N=0, W=0, Y=0, up=0), 0)], ids=str)
def test_adapter_arguments(L, bad, status):
    assert _adapter(L, **bad) == status


def _adapter_back(L, dt=F32, M=4, N=4, K=8, X=P, ldx=8, plan=P, n=2, r=2, down=P, up=P, scale=0, ids=P, S=P, dY=P,
                  lddy=4, dX=P, lddx=8, dd=P, du=P):
    return L.sgemm_emu_adapter_linear_backward(dt, M, N, K, X, ldx, plan, n, r, down, up, scale, ids, S, dY, lddy, dX,
                                               lddx, dd, du, None, 0, None)


@pytest.mark.parametrize("bad,status", [
    (dict(plan=0), ENULL), (dict(plan=P + 8), EINVAL), (dict(S=0), ENULL), (dict(S=P + 4), EINVAL), (dict(dY=0), ENULL),
    (dict(X=0), ENULL), (dict(ids=0), ENULL), (dict(down=0), ENULL), (dict(up=0), ENULL), (dict(lddy=3), EINVAL),
    (dict(lddx=7), EINVAL), (dict(dd=P + 2), EINVAL), (dict(du=P + 2), EINVAL), (dict(n=-1), EINVAL)], ids=str)
def test_adapter_backward_arguments(L, bad, status):
    assert _adapter_back(L, **bad) == status


def test_valid_calls_without_gpu_report_arch(L):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    assert _gated(L) == _gated_back(L) == _adapter(L) == _adapter_back(L) == EARCH
    assert L.sgemm_emu_gated_linear_workspace(F32, 4, 4, 8, P, 8, P, 8, None, None) == EARCH
    assert L.sgemm_emu_gated_linear_backward_workspace(F32, 4, 4, 8) == EARCH
    assert L.sgemm_emu_adapter_linear_workspace(F32, 4, 4, 8, P, 8, P, 8, None, 2, 2, P, None) == EARCH
    assert L.sgemm_emu_adapter_linear_backward_workspace(F32, 4, 4, 8, 2, 2) == EARCH
    assert L.sgemm_emu_plan_weight(F32, 4, 4, P, 4, 0, P, None) == EARCH


def test_workspace_queries_refuse(L):
    assert L.sgemm_emu_gated_linear_workspace(F32, -4, 4, 8, P, 8, P, 8, None, None) == EINVAL
    assert L.sgemm_emu_gated_linear_backward_workspace(3, 4, 4, 8) == EINVAL
    assert L.sgemm_emu_adapter_linear_workspace(F32, 4, 4, 8, P, 8, P, 8, None, -2, 2, P, None) == EINVAL
    assert L.sgemm_emu_adapter_linear_backward_workspace(F32, 4, 4, 8, 2, -2) == EINVAL


def test_few_rows(L):
    assert L.sgemm_emu_few_rows() >= 1


def test_tensor_functions_refuse_host_tensors_and_wrong_types():
    from fp32_emulated_gemm_amd.adapters import adapter_linear
    from fp32_emulated_gemm_amd.gated import gated_linear
    x, w = torch.zeros(3, 8), torch.zeros(6, 8)
    a, b, ids = torch.zeros(2, 4, 8), torch.zeros(2, 6, 4), torch.zeros(3, dtype=torch.int32)
    if torch.cuda.is_available():
        pytest.skip("the refusals on a GPU are tested there")
    for call in (lambda: gated_linear(x.double(), w.double()), lambda: gated_linear("x", w),
                 lambda: adapter_linear(x.half(), w, a, b, ids)):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(ValueError):
        gated_linear(x, w, gate="tanh")
