"""The example that trains and serves a gated block with adapters."""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


# a served output passes two roundings to bfloat16 (h, then y), whose terms are of the outputs'
# size or below; float32 leaves the sums' own errors
@pytest.mark.parametrize("dtype,tol", [("bf16", 2.0 ** -6), ("f32", 1e-5)])
def test_trains_and_serves(dtype, tol):
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import adapted_block
    finally:
        sys.path.pop(0)
    first, last, worst = adapted_block.main(["--dtype", dtype, "--features", "192", "--hidden", "320", "--rows", "300",
                                             "--steps", "20", "--tokens", "3", "--batch", "9"])
    assert last < first
    assert worst < tol
