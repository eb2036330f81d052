"""A gated feed-forward block with low-rank adapters: several users' adapters are
fine-tuned together beside fixed down-projection weights, then their single tokens are
served in one call each step.

    python examples/adapted_block.py [--dtype bf16|f32] [--features 512] [--hidden 1408]
                                     [--adapters 4] [--rank 8] [--steps 30]

    y = x + down(h) + scale[i] up_i (down_i h),   h = silu(x Wg^T) * (x Wu^T)

The gated projection is GatedLinear, trained along with the adapters; the down projection is
AdapterLinear, its weight fixed.  The data are packed sequences, two of each user, whose targets
are the block's own first outputs moved by a direction of that user's.  Prints the loss as it
falls and the served tokens' difference from a float64 evaluation of the same weights; needs an
MI355X.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from fp32_emulated_gemm_amd.adapters import AdapterLinear  # noqa: E402
from fp32_emulated_gemm_amd.gated import GatedLinear  # noqa: E402


class AdaptedBlock(torch.nn.Module):
    def __init__(self, features, hidden, adapters, rank, dtype, device="cuda"):
        super().__init__()
        self.gated = GatedLinear(features, hidden, bias=False, gate="silu", device=device, dtype=dtype)
        self.down = AdapterLinear(hidden, features, adapters, rank, alpha=rank, bias=False, device=device, dtype=dtype)
        self.down.fix_weights()

    def forward(self, x, ids):
        return x + self.down(self.gated(x), ids)

    def reference(self, x, ids):
        """The same weights in float64."""
        x = x.double()
        z = x @ self.gated.weight.double().t()
        F = z.shape[1] // 2
        h = torch.nn.functional.silu(z[:, :F]) * z[:, F:]
        y = x + h @ self.down.weight.double().t()
        for i in range(self.down.adapters):
            rows = ids == i
            low = h[rows] @ self.down.down[i].double().t() * self.down.scale[i].double()
            y[rows] += low @ self.down.up[i].double().t()
        return y


def train(block, steps, rows, seed):
    """Fine-tunes on packed sequences of all users; returns the first and the last loss."""
    features, n = block.down.out_features, block.down.adapters
    dtype, g = block.gated.weight.dtype, torch.Generator("cuda").manual_seed(seed)
    ids = (torch.arange(rows, device="cuda") * (2 * n) // rows % n).int()        # two sequences of each user
    x = torch.randn(rows, features, generator=g, device="cuda").to(dtype)
    direction = torch.randn(n, features, generator=g, device="cuda")
    with torch.no_grad():
        target = block(x, ids).float() + 0.1 * x.float()[:, :1] * direction[ids.long()]
    optimizer = torch.optim.Adam(block.parameters(), lr=2e-3)
    losses = []
    for step in range(steps):
        loss = (block(x, ids).float() - target).square().mean()
        optimizer.zero_grad()
        loss.backward()
        optimizer.step()
        losses.append(loss.item())
        if step % 10 == 0 or step == steps - 1:
            print(f"step {step}: loss {losses[-1]:.4f}", flush=True)
    return losses[0], losses[-1]


def serve(block, tokens, batch, seed):
    """Decodes `tokens` single tokens of `batch` requests, each with its own adapter (or none);
    returns the largest difference from float64, relative to the largest output."""
    features, n = block.down.out_features, block.down.adapters
    dtype, g = block.gated.weight.dtype, torch.Generator("cuda").manual_seed(seed)
    block.gated.fix_weights()
    x = torch.randn(batch, features, generator=g, device="cuda").to(dtype)
    worst = 0.0
    with torch.no_grad():
        for _ in range(tokens):
            ids = torch.randint(-1, n, (batch,), generator=g, device="cuda", dtype=torch.int32)
            y, want = block(x, ids), block.reference(x, ids)
            worst = max(worst, ((y.double() - want).abs().max() / want.abs().max()).item())
            x = torch.nn.functional.layer_norm(y.float(), (features,)).to(dtype)
    return worst


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--dtype", choices=("bf16", "f32"), default="bf16")
    p.add_argument("--features", type=int, default=512)
    p.add_argument("--hidden", type=int, default=1408)
    p.add_argument("--adapters", type=int, default=4)
    p.add_argument("--rank", type=int, default=8)
    p.add_argument("--rows", type=int, default=1024)
    p.add_argument("--steps", type=int, default=30)
    p.add_argument("--tokens", type=int, default=4)
    p.add_argument("--batch", type=int, default=16)
    p.add_argument("--seed", type=int, default=0)
    a = p.parse_args(argv)
    torch.manual_seed(a.seed)
    dtype = torch.bfloat16 if a.dtype == "bf16" else torch.float32
    block = AdaptedBlock(a.features, a.hidden, a.adapters, a.rank, dtype)
    first, last = train(block, a.steps, a.rows, a.seed)
    worst = serve(block, a.tokens, a.batch, a.seed + 1)
    print(f"loss {first:.4f} -> {last:.4f}; {a.tokens} tokens of {a.batch} requests served, "
          f"largest difference from float64 {worst:.2e}", flush=True)
    return first, last, worst


if __name__ == "__main__":
    main()
