"""The experts' operators at the ends of what they take: no experts at all, and products
of more workgroups than one dimension of a launch holds."""
import pytest

from test_gpu_experts import _check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,k", [(31, 2), (70, 2), (700, 3)])
@pytest.mark.parametrize("gate,bias", [(None, True), ("silu", True), ("gelu", False), ("relu", True)])
def test_no_experts(dtype, T, k, gate, bias):
    """Rows of no expert alone: outputs and gradients are zeros, whatever the number of rows."""
    _check(dtype, T, k, 0, 34, 40, gate, bias, "none")
