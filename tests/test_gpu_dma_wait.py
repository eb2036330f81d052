"""The pipelined N x K plane kernels wait for their LDS copies whatever loads the
compiler makes of an unaligned A: repeated products give the same bits."""
import numpy as np
import pytest

from test_gpu_gemm import _rng, fe, run  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,N,K", [(1030, 300, 90), (1030, 300, 1022), (2050, 2050, 129)],
                         ids=lambda v: str(v))
def test_unaligned_a_repeats_bit_for_bit(fe, M, N, K):  # noqa: F811
    """Rows of A that are no multiple of 16 bytes: element loads beside the copies."""
    g = _rng(K)
    A = g.standard_normal((M, K)).astype(np.float32)
    B = g.standard_normal((K, N)).astype(np.float32)
    first = run(fe, A, B, entry="fused_ws")
    for i in range(60):
        again = run(fe, A, B, entry="fused_ws")
        assert np.array_equal(first.view(np.uint32), again.view(np.uint32)), f"repeat {i} differs"
