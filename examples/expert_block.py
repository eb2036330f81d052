"""A feed-forward layer of experts behind a router: trained on packed sequences with
padding, then served with weights of 4 bits, a few tokens at a time, from a graph.

    python examples/expert_block.py [--dtype bf16|f32] [--features 256] [--hidden 384]
                                    [--experts 8] [--choices 2] [--steps 30]

    ids, weights = the choices largest of softmax(x R^T), renormalised
    y[t] = x[t] + sum over j of weights[t, j] down_e(silu(gate_e x) * up_e x),  e = ids[t, j]

The router is a plain linear layer whose gradient comes through the weights.  The
targets are the block's own first outputs moved by a direction of each token's class.
Prints the loss as it falls, and the served tokens' difference from a float64 evaluation
of the 4-bit weights; needs an MI355X.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from fp32_emulated_gemm_amd.experts import ExpertFeedForward  # noqa: E402
from fp32_emulated_gemm_amd.quant4 import Quant4ExpertFeedForward  # noqa: E402


class ExpertBlock(torch.nn.Module):
    def __init__(self, features, hidden, experts, choices, dtype, device="cuda"):
        super().__init__()
        self.router = torch.nn.Linear(features, experts, bias=False, device=device)
        self.layer = ExpertFeedForward(features, hidden, experts, device=device, dtype=dtype)
        self.choices = choices

    def route(self, x, padding=None):
        """ids [T, k] (-1 for padded tokens) and weights [T, k] of a token's experts."""
        best = torch.softmax(self.router(x.float()), dim=1).topk(self.choices, dim=1)
        ids = best.indices.int()
        if padding is not None:
            ids = torch.where(padding.unsqueeze(1), -1, ids)
        return ids, best.values / best.values.sum(dim=1, keepdim=True)

    def forward(self, x, padding=None):
        ids, weights = self.route(x, padding)
        return x + self.layer(x, ids, weights)


def train(block, steps, rows, seed):
    """Trains on packed sequences of which one token in eight is padding; returns the first and the last loss."""
    features, dtype = block.layer.features, block.layer.up.dtype
    g = torch.Generator("cuda").manual_seed(seed)
    x = torch.randn(rows, features, generator=g, device="cuda").to(dtype)
    padding = torch.arange(rows, device="cuda") % 8 == 7
    direction = torch.randn(2, features, generator=g, device="cuda")
    with torch.no_grad():
        target = block(x, padding).float() + 0.2 * direction[(x[:, 0] > 0).long()]
    optimizer = torch.optim.Adam(block.parameters(), lr=2e-3)
    losses = []
    for step in range(steps):
        loss = (block(x, padding).float() - target)[~padding].square().mean()
        optimizer.zero_grad()
        loss.backward()
        optimizer.step()
        losses.append(loss.item())
        if step % 10 == 0 or step == steps - 1:
            print(f"step {step}: loss {losses[-1]:.4f}", flush=True)
    return losses[0], losses[-1]


def reference(block, served, x):
    """The served block in float64, token by token."""
    ids, weights = block.route(x)
    up, down = (served._held(name).dequantize().double() for name in ("up", "down"))
    x = x.double()
    y = x.clone()
    for t in range(x.shape[0]):
        for j, e in enumerate(ids[t].tolist()):
            z = up[e] @ x[t]
            F = z.shape[0] // 2
            y[t] += weights[t, j].double() * (down[e] @ (torch.nn.functional.silu(z[:F]) * z[F:]))
    return y


def serve(block, tokens, batch, group, seed):
    """`tokens` steps of `batch` tokens through the layer in 4 bits, replayed from one graph; returns the
    largest difference from float64, relative to the largest output."""
    served = Quant4ExpertFeedForward.from_experts(block.layer, group)
    g = torch.Generator("cuda").manual_seed(seed)
    x = torch.zeros(batch, block.layer.features, device="cuda", dtype=block.layer.up.dtype)

    def step():
        ids, weights = block.route(x)
        return x + served(x, ids, weights)

    worst = 0.0
    with torch.no_grad():
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y = step()
        for _ in range(tokens):
            x.copy_(torch.randn(x.shape, generator=g, device="cuda"))
            graph.replay()
            want = reference(block, served, x)
            worst = max(worst, ((y.double() - want).abs().max() / want.abs().max()).item())
    return worst


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--dtype", choices=("bf16", "f32"), default="bf16")
    p.add_argument("--features", type=int, default=256)
    p.add_argument("--hidden", type=int, default=384)
    p.add_argument("--experts", type=int, default=8)
    p.add_argument("--choices", type=int, default=2)
    p.add_argument("--rows", type=int, default=1024)
    p.add_argument("--steps", type=int, default=30)
    p.add_argument("--tokens", type=int, default=4)
    p.add_argument("--batch", type=int, default=16)
    p.add_argument("--group", type=int, default=64)
    p.add_argument("--seed", type=int, default=0)
    a = p.parse_args(argv)
    torch.manual_seed(a.seed)
    dtype = torch.bfloat16 if a.dtype == "bf16" else torch.float32
    block = ExpertBlock(a.features, a.hidden, a.experts, a.choices, dtype)
    first, last = train(block, a.steps, a.rows, a.seed)
    worst = serve(block, a.tokens, a.batch, a.group, a.seed + 1)
    print(f"loss {first:.4f} -> {last:.4f}; {a.tokens} steps of {a.batch} tokens served in 4 bits, "
          f"largest difference from float64 {worst:.2e}", flush=True)
    return first, last, worst


if __name__ == "__main__":
    main()
