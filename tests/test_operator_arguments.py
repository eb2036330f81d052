"""Checks of the operators' arguments that need no GPU: what the tensor functions
make of strides, which layouts of a weight they take, sizes whose products wrap."""
import pytest
import torch

EINVAL, EARCH = -1, -3
P = 0x10000   # any nonzero, 256-byte aligned address: never dereferenced on these paths


@pytest.fixture(scope="module")
def L():
    from fp32_emulated_gemm_amd import ops
    return ops.ops_lib()


@pytest.mark.parametrize("held", [None, "laid out"])
def test_a_plan_stands_for_its_own_operator_only(held):
    """The two layouts have one shape and type, whether the forward's rows are copied or lie."""
    from fp32_emulated_gemm_amd.ops import WeightPlan
    w = torch.zeros(6, 8)
    for gated in (True, False):
        plan = WeightPlan.__new__(WeightPlan)
        plan.dtype, plan.shape, plan.device, plan.gated = w.dtype, (6, 8), w.device, gated
        plan.forward, plan.backward = held, None
        plan.check(w, gated=gated)
        with pytest.raises(ValueError):
            plan.check(w, gated=not gated)
        with pytest.raises(ValueError):
            plan.check(w[:4], gated=gated)


@pytest.mark.parametrize("rows,cols,stride,copied", [
    (1, 16, (8_392_704, 1), False),      # the last token of a long prompt: one row, whatever its stride
    (1, 16, (0, 1), False), (1, 16, (3, 1), False), (1, 1, (1, 5), False), (1, 16, (16, 2), True),
    (3, 16, (8_392_704, 1), True), (3, 16, (8_388_544, 1), False), (3, 16, (8_388_545, 1), True),
    (3, 16, (16, 1), False), (3, 16, (24, 1), False), (3, 16, (0, 1), True), (3, 16, (8, 1), True),
    (3, 16, (1, 3), True), (3, 1, (1, 1), False), (3, 1, (7, 9), False), (0, 16, (16, 1), False),
    (3, 0, (1, 1), False), (0, 0, (1, 1), False)])
def test_rows_of_any_stride(rows, cols, stride, copied):
    """Rows come with a leading dimension that the library takes, and keep their values."""
    from fp32_emulated_gemm_amd.ops import rows_of
    need = 1 + sum((n - 1) * s for n, s in zip((rows, cols), stride)) if rows and cols else 0
    base = torch.arange(need, dtype=torch.int32)
    t = torch.as_strided(base, (rows, cols), stride)
    got, ld = rows_of(t)
    assert (got is not t) == copied
    assert max(cols, 1) <= ld <= 8_388_544
    assert got.shape == t.shape and torch.equal(got, t)
    if rows and cols:
        again = torch.as_strided(got, (rows, cols), (ld, 1)) if cols > 1 or rows > 1 else got
        assert torch.equal(again, t)


@pytest.mark.parametrize("F", [-2 ** 63, -2 ** 63 + 1, -2 ** 63 + 1000, -1, 2 ** 62, 2 ** 63 - 1, 2 ** 21])
def test_a_width_whose_double_wraps_is_refused(L, F):
    assert L.sgemm_emu_gated_linear_workspace(0, 4, F, 8, P, 8, P, 8, None, None) == EINVAL
    assert L.sgemm_emu_gated_linear_backward_workspace(0, 4, F, 8) == EINVAL
    ld = max(F, 1) if F < 2 ** 23 else 2 ** 22
    assert L.sgemm_emu_gated_linear(0, 4, F, 8, P, 8, P, 8, None, None, 0, P, ld, None, None, 0, None) == EINVAL


@pytest.mark.parametrize("n,r,N,K,fits", [
    (65535, 4194240, 4194240, 4194240, False), (65535, 4194240, 4194240, 0, False), (65535, 1 << 20, 1 << 20, 1, False),
    (65535, 256, 16384, 16384, True), (1, 4194240, 4194240, 4194240, True), (65535, 4194240, 0, 0, True),
    (0, 4194240, 4194240, 4194240, True)])
def test_banks_whose_bytes_wrap_are_refused(L, n, r, N, K, fits):
    """A workspace's size adds up the banks' copies and the partial sums of their gradients."""
    for dtype in (0, 1):
        for got in (L.sgemm_emu_adapter_linear_workspace(dtype, 4, N, K, P, max(K, 1), P, max(K, 1), None, n, r, P, None),
                    L.sgemm_emu_adapter_linear_backward_workspace(dtype, 4, N, K, n, r)):
            if not fits:
                assert got == EINVAL
            elif torch.cuda.is_available():
                assert 0 <= got < 2 ** 62
            else:
                assert got == EARCH
