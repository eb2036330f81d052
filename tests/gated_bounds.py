"""Bounds of the bfloat16 gated projection's gradients with its pre-activations kept
in 32 bits: ops_reference's bounds of the same operands as float32 tensors (the
errors of the sums and of the gate), and on top of them what is rounded to
bfloat16, dZ as an operand of dX and dW, and each output once."""
import torch

import ops_reference as ref


def gated_gradients(x, w, bias, gate, dh):
    """{name: (reference, bound)} of dX, dW, dbias; CPU bfloat16 tensors."""
    wide = ref.gated(x.float(), w.float(), None if bias is None else bias.float(), gate, dh.float())
    X, W, F = x.double(), w.double(), w.shape[0] // 2
    z = X @ W.T + (0 if bias is None else bias.double())
    a, d = ref.act64(z[:, :F], gate)
    dz = torch.cat((dh.double() * z[:, F:] * d, dh.double() * a), 1).abs()
    operand = {"dx": dz @ W.abs(), "dw": dz.T @ X.abs(), "db": 0.0}
    return {name: (wide[name][0], wide[name][1] + ref.SLACK * ref.BF * (operand[name] + wide[name][0].abs()))
            for name in operand}
