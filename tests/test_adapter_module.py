"""AdapterLinear as a torch module: casts and moves.  No GPU."""
import pytest
import torch


@pytest.mark.parametrize("cast", [lambda m: m.to(torch.bfloat16), lambda m: m.bfloat16(),
                                  lambda m: torch.nn.Sequential(m).to(torch.bfloat16)[0]])
def test_a_cast_leaves_the_scale_in_32_bits(cast):
    """The layer's tensors change their type; the scale, float32 whatever that is, keeps its value
    (here none of bfloat16)."""
    from fp32_emulated_gemm_amd.adapters import AdapterLinear
    m = AdapterLinear(8, 6, adapters=2, rank=3, alpha=16)
    want = m.scale.clone()
    assert (want.bfloat16().float() != want).all()
    m = cast(m)
    assert {t.dtype for t in (m.weight, m.bias, m.down, m.up)} == {torch.bfloat16}
    assert m.scale.dtype == torch.float32 and torch.equal(m.scale, want)
    assert "scale" in dict(m.named_buffers()) and "scale" in m.state_dict()
    assert m.float().scale.dtype == torch.float32 and torch.equal(m.scale, want)
