"""Modules served in 4 bits, on the host: which layers they are made from."""
import pytest

from fp32_emulated_gemm_amd.adapters import AdapterLinear
from fp32_emulated_gemm_amd.linear import Linear
from fp32_emulated_gemm_amd.quant4 import Quant4Linear


def test_layers_that_compute_more_are_refused():
    """A fused activation or adapters would be left out of the served layer without a word."""
    with pytest.raises(ValueError, match="activation"):
        Quant4Linear.from_linear(Linear(8, 6, activation="gelu"))
    with pytest.raises(ValueError, match="adapters"):
        Quant4Linear.from_linear(AdapterLinear(8, 6, 2, 4))
