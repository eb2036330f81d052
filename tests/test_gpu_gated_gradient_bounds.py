"""The bfloat16 gated projection's gradients on the GPU within the bounds of
pre-activations kept in 32 bits."""
import pytest

import ops_reference as ref
from gated_bounds import gated_gradients
from test_gated_gradient_bounds import SIZES
from test_gpu_gated import SHAPES, _inputs, _run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,K,F", SHAPES + SIZES + [(700, 768, 520), (2100, 264, 300)])
def test_gradients(M, K, F):
    x, w, b, dh = _inputs("bf16", M, K, F, True, seed=31)
    got = _run(x, w, b, dh, "silu")
    for name, bound in gated_gradients(x, w, b, "silu", dh).items():
        ref.check(got[name], bound, name)


@pytest.mark.parametrize("gate", ["gelu", "gelu_tanh", "sigmoid"])
@pytest.mark.parametrize("M,K,F", SIZES + [(513, 136, 72)])
def test_gates(gate, M, K, F):
    x, w, b, dh = _inputs("bf16", M, K, F, True, seed=33)
    got = _run(x, w, b, dh, gate)
    for name, bound in gated_gradients(x, w, b, gate, dh).items():
        ref.check(got[name], bound, name)
