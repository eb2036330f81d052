"""Checks of the C ABI of include/sgemm_emu_experts.h that need no GPU: every function
declared, exported and bound, the header's C99 and C++17, workspace sizes, arguments
refused before any HIP call, and the tensor functions' refusals."""
import ctypes
import os
import re
import shutil
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "sgemm_emu_experts.h")
P = 0x10000  # any nonzero, 256-byte aligned address: never dereferenced on these paths
F32, BF16 = 0, 1
EINVAL, ENULL, EARCH = -1, -2, -3
BIG = 1 << 22


def _declared():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    return sorted(set(re.findall(r"^(?:int|int64_t)\s+(\w+)\s*\(", text, flags=re.M)))


@pytest.fixture(scope="module")
def L():
    from fp32_emulated_gemm_amd import experts
    return experts.experts_lib()


def test_declared_exported_and_bound(L):
    import fp32_emulated_gemm_amd as fe
    from fp32_emulated_gemm_amd import experts
    assert _declared() == sorted(experts.EXPERTS_EXPORTS)
    libs = [L]
    if not os.environ.get("SGEMM_EMU_LIB_OVERRIDE"):
        libs.append(ctypes.CDLL(os.path.join(os.path.dirname(os.path.abspath(fe.__file__)),
                                             "libsgemm_emu_serial_lds.so")))
    for lib in libs:
        for name in _declared():
            assert hasattr(lib, name), name
    text = open(HEADER).read()
    assert f"#define SGEMM_EMU_MAX_EXPERTS {experts.SGEMM_EMU_MAX_EXPERTS}\n" in text


def test_header_in_c_and_cxx(tmp_path):
    if shutil.which("gcc") is None or shutil.which("g++") is None:
        pytest.skip("no host C compiler")
    src = tmp_path / "experts.c"
    src.write_text('#include "sgemm_emu_experts.h"\nint main(void) { return SGEMM_EMU_GATE_NONE + 1; }\n')
    inc = os.path.join(ROOT, "include")
    for cc in (["gcc", "-std=c99", "-pedantic"], ["g++", "-std=c++17", "-x", "c++"]):
        subprocess.run([*cc, "-Wall", "-Wextra", "-Werror", "-I", inc, "-c", str(src), "-o", str(tmp_path / "o")],
                       check=True)


def _sort(L, n_pairs=8, n=4, ids=P, offsets=P, pairs=P, places=P, ws=0, ws_bytes=0):
    return L.sgemm_emu_sort_tokens(n_pairs, n, ids, offsets, pairs, places, ws, ws_bytes, None)


@pytest.mark.parametrize("bad,status", [
    (dict(n_pairs=-1), EINVAL), (dict(n_pairs=BIG), EINVAL), (dict(n=-1), EINVAL), (dict(n=1025), EINVAL),
    (dict(ids=0), ENULL), (dict(offsets=0), ENULL), (dict(pairs=0), ENULL), (dict(places=0), ENULL),
    (dict(ids=P + 2), EINVAL), (dict(offsets=P + 1), EINVAL), (dict(n_pairs=100000), ENULL),
    (dict(n_pairs=100000, ws=P, ws_bytes=16), EINVAL), (dict(n_pairs=100000, ws=P + 4, ws_bytes=1 << 20), EINVAL)], ids=str)
def test_sort_arguments(L, bad, status):
    assert _sort(L, **bad) == status


def test_sort_workspace(L):
    for n_pairs, n in ((0, 0), (1, 1024), (4096, 64)):
        assert L.sgemm_emu_sort_tokens_workspace(n_pairs, n) == 0
    assert L.sgemm_emu_sort_tokens_workspace(4097, 63) == 2 * 64 * 4
    for bad in ((-1, 4), (BIG, 4), (4, -1), (4, 1025)):
        assert L.sgemm_emu_sort_tokens_workspace(*bad) == EINVAL


def _gather(L, dt=F32, T=4, k=2, K=8, n=3, X=P, ldx=8, offsets=P, places=P, Xs=P, ldxs=8):
    return L.sgemm_emu_gather_tokens(dt, T, k, K, n, X, ldx, offsets, places, Xs, ldxs, None)


@pytest.mark.parametrize("bad,status", [
    (dict(dt=2), EINVAL), (dict(T=-1), EINVAL), (dict(k=-1), EINVAL), (dict(K=-1), EINVAL), (dict(n=1025), EINVAL),
    (dict(T=1 << 21, k=4), EINVAL), (dict(T=1 << 21, k=1 << 62), EINVAL), (dict(ldx=7), EINVAL), (dict(ldxs=7), EINVAL),
    (dict(ldx=1 << 24), EINVAL), (dict(X=0), ENULL), (dict(Xs=0), ENULL), (dict(offsets=0), ENULL),
    (dict(places=0), ENULL), (dict(X=P + 2), EINVAL), (dict(dt=BF16, X=P + 1), EINVAL), (dict(places=P + 2), EINVAL)], ids=str)
def test_gather_arguments(L, bad, status):
    assert _gather(L, **bad) == status


def _combine(L, dt=F32, T=4, k=2, K=8, Ys=P, ldys=8, places=P, weights=0, Y=P, ldy=8):
    return L.sgemm_emu_combine_tokens(dt, T, k, K, Ys, ldys, places, weights, Y, ldy, None)


@pytest.mark.parametrize("bad,status", [
    (dict(dt=-1), EINVAL), (dict(T=-1), EINVAL), (dict(k=-1), EINVAL), (dict(K=BIG), EINVAL), (dict(ldys=7), EINVAL),
    (dict(ldy=7), EINVAL), (dict(Ys=0), ENULL), (dict(Y=0), ENULL), (dict(places=0), ENULL), (dict(weights=P + 2), EINVAL)],
    ids=str)
def test_combine_arguments(L, bad, status):
    assert _combine(L, **bad) == status


def _combine_back(L, dt=F32, T=4, k=2, K=8, n=3, Ys=P, ldys=8, offsets=P, places=P, weights=0, dY=P, lddy=8, dYs=P,
                  lddys=8, dw=P):
    return L.sgemm_emu_combine_tokens_backward(dt, T, k, K, n, Ys, ldys, offsets, places, weights, dY, lddy, dYs, lddys,
                                               dw, None)


@pytest.mark.parametrize("bad,status", [
    (dict(dt=2), EINVAL), (dict(T=-1), EINVAL), (dict(n=-1), EINVAL), (dict(Ys=0), ENULL), (dict(dY=0), ENULL),
    (dict(offsets=0), ENULL), (dict(places=0), ENULL), (dict(lddy=7), EINVAL), (dict(lddys=7), EINVAL),
    (dict(dw=P + 1), EINVAL), (dict(weights=P + 1), EINVAL)], ids=str)
def test_combine_backward_arguments(L, bad, status):
    assert _combine_back(L, **bad) == status


def _expert(L, dt=F32, rows=8, N=4, K=8, n=3, X=P, ldx=8, W=P, bias=0, gate=-1, offsets=P, H=P, ldh=4, Z=0):
    return L.sgemm_emu_expert_linear(dt, rows, N, K, n, X, ldx, W, bias, gate, offsets, H, ldh, Z, None)


@pytest.mark.parametrize("bad,status", [
    (dict(dt=2), EINVAL), (dict(rows=-1), EINVAL), (dict(rows=BIG), EINVAL), (dict(N=-1), EINVAL), (dict(K=BIG), EINVAL),
    (dict(n=-1), EINVAL), (dict(n=1025), EINVAL), (dict(n=1000, N=1 << 21, K=1 << 21, ldx=1 << 21), EINVAL),
    (dict(gate=5), EINVAL), (dict(gate=-2), EINVAL), (dict(gate=0, N=5), EINVAL), (dict(ldx=7), EINVAL),
    (dict(ldh=3), EINVAL), (dict(X=0), ENULL), (dict(W=0), ENULL), (dict(H=0), ENULL), (dict(offsets=0), ENULL),
    (dict(W=P + 2), EINVAL), (dict(dt=BF16, W=P + 1), EINVAL), (dict(bias=P + 2), EINVAL), (dict(offsets=P + 2), EINVAL),
    (dict(gate=0, Z=P + 8), EINVAL), (dict(Z=P), EINVAL)], ids=str)
def test_expert_arguments(L, bad, status):
    assert _expert(L, **bad) == status


def _expert_back(L, dt=F32, rows=8, N=4, K=8, n=3, X=P, ldx=8, W=P, Z=P, gate=0, offsets=P, dH=P, lddh=4, dX=P, lddx=8,
                 dW=P, db=P, ws=P, ws_bytes=1 << 30):
    return L.sgemm_emu_expert_linear_backward(dt, rows, N, K, n, X, ldx, W, Z, gate, offsets, dH, lddh, dX, lddx, dW, db,
                                              ws, ws_bytes, None)


@pytest.mark.parametrize("bad,status", [
    (dict(dt=2), EINVAL), (dict(rows=-1), EINVAL), (dict(n=1025), EINVAL), (dict(gate=9), EINVAL), (dict(N=3), EINVAL),
    (dict(X=0), ENULL), (dict(W=0), ENULL), (dict(Z=0), ENULL), (dict(dH=0), ENULL), (dict(offsets=0), ENULL),
    (dict(lddx=7), EINVAL), (dict(lddh=1), EINVAL), (dict(Z=P + 4), EINVAL), (dict(dW=P + 2), EINVAL), (dict(ws=0), ENULL),
    (dict(ws=P + 8), EINVAL), (dict(ws_bytes=100), EINVAL)], ids=str)
def test_expert_backward_arguments(L, bad, status):
    assert _expert_back(L, **bad) == status


def test_expert_backward_workspace(L):
    ask = L.sgemm_emu_expert_linear_backward_workspace
    assert ask(F32, 8, 4, 8, 3, -1, 0) == 0
    # halves of dZ's rows are padded to 128 columns; a row of sums for each tile of 64 rows
    assert ask(F32, 8, 4, 8, 3, 0, 0) == 8 * 256 * 4
    assert ask(BF16, 8, 4, 8, 3, 0, 1) == 8 * 256 * 2 + 256
    # few tiles and many rows: pieces of 256 rows
    assert ask(F32, 4096, 128, 64, 4, -1, 0) == (4096 // 256 + 4) * 128 * 64 * 4
    assert ask(F32, 4096, 4096, 4096, 4, -1, 0) == 0
    for bad in ((2, 8, 4, 8, 3, 0, 0), (F32, -1, 4, 8, 3, 0, 0), (F32, 8, 5, 8, 3, 0, 0), (F32, 8, 4, 8, 1025, 0, 0),
                (F32, 8, 4, 8, 3, 7, 0)):
        assert ask(*bad) == EINVAL


def _pack(L, n=1, N=4, K=8, group=32, q=P, scale=P, zero=0, packed=P):
    return L.sgemm_emu_quant4_pack(n, N, K, group, q, scale, zero, packed, None)


@pytest.mark.parametrize("bad,status", [
    (dict(n=-1), EINVAL), (dict(n=1025), EINVAL), (dict(N=-1), EINVAL), (dict(K=BIG), EINVAL), (dict(group=16), EINVAL),
    (dict(group=0), EINVAL), (dict(q=0), ENULL), (dict(scale=0), ENULL), (dict(packed=0), ENULL),
    (dict(scale=P + 2), EINVAL), (dict(packed=P + 8), EINVAL)], ids=str)
def test_pack_arguments(L, bad, status):
    assert _pack(L, **bad) == status


def test_quant4_sizes(L):
    # tiles of 16 rows by 128 columns in 1 KB, scales and zeros for 16 rows and 128 columns up, spare bytes
    assert L.sgemm_emu_quant4_bytes(1, 16, 128, 128, 0) == 1024 + 64 + 64
    assert L.sgemm_emu_quant4_bytes(1, 16, 128, 32, 1) == 1024 + 4 * 64 + 64 + 64
    assert L.sgemm_emu_quant4_bytes(3, 17, 129, 64, 1) == 3 * (4 * 1024 + 4 * 32 * 4 + 128 + 64)
    for bad in ((-1, 4, 4, 32, 0), (1, -1, 4, 32, 0), (1, 4, BIG, 32, 0), (1, 4, 4, 33, 0), (1025, 4, 4, 32, 0)):
        assert L.sgemm_emu_quant4_bytes(*bad) == EINVAL
    ask = L.sgemm_emu_quant4_linear_workspace
    assert ask(BF16, 64, 100, 100, 1, 128, 0) == 0
    assert ask(BF16, 65, 100, 100, 1, 128, 0) == -(-100 * 100 * 2 // 256) * 256
    assert ask(F32, 128, 10, 10, 8, 128, 0) == 0
    assert ask(BF16, 65, 100, 100, 1, 100, 0) == EINVAL


def _quant4(L, dt=F32, rows=4, N=4, K=8, n=1, group=32, zeros=0, X=P, ldx=8, packed=P, bias=0, gate=-1, offsets=0, H=P,
            ldh=4, ws=0, ws_bytes=0):
    return L.sgemm_emu_quant4_linear(dt, rows, N, K, n, group, zeros, X, ldx, packed, bias, gate, offsets, H, ldh, ws,
                                     ws_bytes, None)


@pytest.mark.parametrize("bad,status", [
    (dict(dt=3), EINVAL), (dict(rows=-1), EINVAL), (dict(N=-2), EINVAL), (dict(n=2), EINVAL), (dict(group=64 + 1), EINVAL),
    (dict(X=0), ENULL), (dict(packed=0), ENULL), (dict(H=0), ENULL), (dict(packed=P + 4), EINVAL), (dict(ldx=7), EINVAL),
    (dict(gate=6), EINVAL), (dict(gate=0, N=3), EINVAL), (dict(offsets=P + 2), EINVAL), (dict(rows=65), ENULL),
    (dict(rows=65, ws=P, ws_bytes=8), EINVAL)], ids=str)
def test_quant4_arguments(L, bad, status):
    assert _quant4(L, **bad) == status


def test_quantize_arguments(L):
    call = L.sgemm_emu_quant4_quantize
    assert call(2, 1, 4, 8, 32, P, P, P, 0, None) == EINVAL
    assert call(F32, 1, 4, 8, 31, P, P, P, 0, None) == EINVAL
    assert call(F32, 1, 4, 8, 32, 0, P, P, 0, None) == ENULL
    assert call(F32, 1, 4, 8, 32, P, 0, P, 0, None) == ENULL
    assert call(F32, 1, 4, 8, 32, P, P, 0, 0, None) == ENULL
    assert call(F32, 1, 4, 8, 32, P + 2, P, P, 0, None) == EINVAL
    assert L.sgemm_emu_quant4_unpack(F32, 1, 4, 8, 32, 0, P + 8, P, None) == EINVAL
    assert L.sgemm_emu_quant4_unpack(F32, 1, 4, 8, 32, 0, P, 0, None) == ENULL


@pytest.mark.skipif(torch.cuda.is_available(), reason="valid calls would run")
def test_valid_calls_stop_at_the_device(L):
    for status in (_sort(L), _gather(L), _combine(L), _combine_back(L), _expert(L), _expert_back(L), _pack(L), _quant4(L)):
        assert status == EARCH


# ---------------------------------------------------------------- the tensor functions

def _order(T=4, k=2, n=3):
    from fp32_emulated_gemm_amd.experts import ExpertOrder
    return ExpertOrder(torch.zeros(n + 1, dtype=torch.int32), torch.zeros(T * k, dtype=torch.int32),
                       torch.zeros(T, k, dtype=torch.int32), n)


def test_tensor_functions_refuse():
    """Wrong types, and tensors that lie on the host."""
    from fp32_emulated_gemm_amd import experts, quant4
    ids = torch.zeros(4, 2, dtype=torch.int32)
    with pytest.raises(TypeError):
        experts.sort_tokens([[0, 1]], 4)
    with pytest.raises(ValueError):
        experts.sort_tokens(ids.view(2, 2, 2), 4)
    with pytest.raises((TypeError, ValueError)):
        experts.sort_tokens(ids.long(), 4)
    with pytest.raises((ValueError, RuntimeError)):
        experts.sort_tokens(ids, 4)
    for call in (lambda o: experts.gather_tokens(torch.zeros(4, 8), o), lambda o: experts.combine_tokens(torch.zeros(8, 8), o),
                 lambda o: experts.expert_linear(torch.zeros(8, 8), torch.zeros(3, 4, 8), o)):
        with pytest.raises(TypeError):
            call(ids)
        with pytest.raises((ValueError, RuntimeError)):
            call(_order())
    with pytest.raises(TypeError):
        quant4.quant4_linear(torch.zeros(4, 8), torch.zeros(4, 8))
    with pytest.raises(TypeError):
        quant4.pack([1], torch.zeros(1))
    with pytest.raises(ValueError):
        quant4.pack(torch.zeros(4, 8, dtype=torch.uint8), torch.zeros(4, 1), group=48)
    with pytest.raises(ValueError):
        quant4.pack(torch.zeros(8, dtype=torch.uint8), torch.zeros(1))
    with pytest.raises(TypeError):
        quant4.quantize(torch.zeros(4, 8, dtype=torch.float64))
    with pytest.raises(ValueError):
        quant4.quantize(torch.zeros(4))


def test_gate_codes():
    from fp32_emulated_gemm_amd.experts import SGEMM_EMU_GATE_NONE, gate_code
    assert gate_code(None, 5) == SGEMM_EMU_GATE_NONE
    assert [gate_code(g, 4) for g in ("silu", "gelu", "gelu_tanh", "sigmoid", "relu")] == [0, 1, 2, 3, 4]
    with pytest.raises(ValueError):
        gate_code("swish", 4)
    with pytest.raises(ValueError):
        gate_code("silu", 5)


def test_modules_hold_their_parameters():
    """Shapes, initial values and copies of the modules, on the host."""
    from fp32_emulated_gemm_amd.experts import ExpertFeedForward
    m = ExpertFeedForward(6, 10, 3, bias=True, gate="gelu", dtype=torch.bfloat16)
    assert [tuple(p.shape) for p in m.parameters()] == [(3, 20, 6), (3, 6, 10), (3, 20), (3, 6)]
    assert all(p.dtype == torch.bfloat16 for p in m.parameters())
    assert float(m.up.abs().max()) <= 6 ** -0.5 and float(m.up_bias.abs().max()) == 0
    assert "experts=3" in repr(m)
    with pytest.raises(ValueError):
        ExpertFeedForward(6, 10, 3, gate="none")
