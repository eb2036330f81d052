"""The example of a routed layer of experts runs, its gradients are those of float64,
and its served tokens agree with float64."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_runs(dtype):
    import expert_block
    first, last, worst = expert_block.main(["--dtype", dtype, "--features", "72", "--hidden", "40", "--rows", "96",
                                            "--steps", "2", "--tokens", "2", "--batch", "5", "--group", "32"])
    assert first == first and last == last
    # three rounded tensors on the way of a bfloat16 token, and its output; float32: two sums of at most
    # 72 terms of 4-bit values, whose offset by 16 makes a term up to 32 of its own steps
    assert worst <= (4 * 2.0 ** -8 if dtype == "bf16" else 2 * 2 * 72 * 2.0 ** -24 * 32)


def test_gradients():
    """Of the router through the weights, and of the experts, against the same block in float64."""
    import expert_block
    torch.manual_seed(1)
    block = expert_block.ExpertBlock(24, 16, 4, 2, torch.float32)
    x = torch.randn(40, 24, device="cuda")
    padding = torch.arange(40, device="cuda") % 8 == 7
    block(x, padding).square().sum().backward()
    R, up, down = (p.detach().double().requires_grad_(True) for p in (block.router.weight, block.layer.up, block.layer.down))
    ids, _ = block.route(x, padding)
    x64 = x.double()
    chance = torch.softmax(x64 @ R.T, 1)
    total = 0
    for t in range(40):
        y = x64[t]
        if not padding[t]:
            picked = chance[t, ids[t].long()]
            for j, e in enumerate(ids[t].tolist()):
                z = up[e] @ x64[t]
                y = y + picked[j] / picked.sum() * (down[e] @ (torch.nn.functional.silu(z[:16]) * z[16:]))
        total = total + y.square().sum()
    total.backward()
    for got, want in ((block.router.weight.grad, R.grad), (block.layer.up.grad, up.grad), (block.layer.down.grad, down.grad)):
        # chains of sums of at most 40 terms in 32 bits
        assert (got.double() - want).abs().max() <= 4 * 2 * 40 * 2.0 ** -24 * want.abs().max()
