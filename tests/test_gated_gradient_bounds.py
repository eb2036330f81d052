"""That the bounds in gated_bounds tell pre-activations kept in 32 bits from rounded
ones: the gradients' formulas on the CPU, with Z rounded either way.  No GPU.

dbias sums M rows, so rounding Z to bfloat16 moves it by about sqrt(M) 2^-10 of a row's
dZ; its bound grows like M (2 K + 2 M) 2^-24 (the worst sums).  The sizes keep the
second below 0.6 of the first."""
import pytest
import torch

import ops_reference as ref
from gated_bounds import gated_gradients


SIZES = [(65, 16, 32), (130, 16, 40), (257, 8, 136)]


def _gradients(x, w, b, gate, dh, kept):
    """In float64 from Z rounded to `kept`, dZ and the outputs rounded to bfloat16."""
    X, W, F = x.double(), w.double(), w.shape[0] // 2
    z = (X @ W.T + b.double()).to(kept).double()
    a, d = ref.act64(z[:, :F], gate)
    dz = torch.cat((dh.double() * z[:, F:] * d, dh.double() * a), 1)
    low = dz.to(torch.bfloat16).double()
    out = {"dx": low @ W, "dw": low.T @ X, "db": dz.sum(0)}
    return {name: v.to(torch.bfloat16) for name, v in out.items()}


@pytest.mark.parametrize("gate", ["silu", "gelu", "gelu_tanh", "sigmoid"])
@pytest.mark.parametrize("M,K,F", SIZES)
def test_bounds_tell_32_bits_from_16(M, K, F, gate):
    g = torch.Generator().manual_seed(M)
    x, dh = (torch.randn(M, n, generator=g).bfloat16() for n in (K, F))
    w = (torch.randn(2 * F, K, generator=g) * K ** -0.5).bfloat16()
    b = (torch.randn(2 * F, generator=g) * 0.2).bfloat16()
    bounds = gated_gradients(x, w, b, gate, dh)
    loose = ref.gated(x, w, b, gate, dh)
    for name, got in _gradients(x, w, b, gate, dh, torch.float32).items():
        ref.check(got, bounds[name], name)
    rounded = _gradients(x, w, b, gate, dh, torch.bfloat16)
    with pytest.raises(AssertionError):
        ref.check(rounded["db"], bounds["db"], "db")
    for name, got in rounded.items():         # the wider bounds of ops_reference let it pass
        ref.check(got, loose[name], name)
