"""64-bit definitions of the gated projection and the adapter layer, with the
elementwise error bounds that the GPU tests hold the kernels to.

Bounds, derived from the arithmetic and not from results (u = 2^-24):
  a K-term product summed in FP32, from the nine BF16 products, the FP32 matrix
  instruction or exact bfloat16 products: 2 K u sum|a b|  (the elementwise
  criterion of the GEMM tests); a sum of T terms likewise;
  one more FP32 operation: u of its result;
  act, act': (16 + 4 |z|) u of the result's scale (the exponent of exp(-z) is
  rounded: |z| u relative; the rest is a few roundings);
  an output or operand rounded to bfloat16 (8 significant bits): 2^-8 of its value;
  errors of operands propagate with the derivatives' bounds (D, D2 below).
"""
import math

import torch

U = 2.0 ** -24
BF = 2.0 ** -8
TINY = 2.0 ** -120
SLACK = 1.01            # second-order terms

# bounds of |act'|, |act''| over the reals (relu: away from its corner)
D = {"silu": 1.1, "gelu": 1.13, "gelu_tanh": 1.13, "sigmoid": 0.25, "relu": 1.0}
D2 = {"silu": 0.5, "gelu": 0.8, "gelu_tanh": 0.81, "sigmoid": 0.1, "relu": 0.0}


def act64(z, gate):
    """act(z), act'(z) in float64."""
    if gate == "silu":
        s = torch.sigmoid(z)
        return z * s, s * (1 + z * (1 - s))
    if gate == "gelu":
        cdf = torch.special.ndtr(z)
        return z * cdf, cdf + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if gate == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z ** 3))
        return 0.5 * z * (1 + t), 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    if gate == "sigmoid":
        s = torch.sigmoid(z)
        return s, s * (1 - s)
    return torch.clamp(z, min=0), (z > 0).double()


def _out(err, ref, bf16):
    return SLACK * (err + (BF * ref.abs() if bf16 else U * ref.abs())) + TINY


def gated(x, w, bias, gate, dh=None):
    """{name: (reference, bound)} of H (and dX, dW, dbias with dh); CPU tensors of one type."""
    bf16 = x.dtype == torch.bfloat16
    X, W = x.double(), w.double()
    F, K = w.shape[0] // 2, x.shape[1]
    z = X @ W.T
    ez = 2 * K * U * (X.abs() @ W.abs().T)
    if bias is not None:
        z = z + bias.double()
        ez = ez + U * z.abs()
    zg, zu, eg, eu = z[:, :F], z[:, F:], ez[:, :F], ez[:, F:]
    a, d = act64(zg, gate)
    ea = D[gate] * eg + (16 + 4 * zg.abs()) * U * a.abs()
    h = a * zu
    out = {"h": (h, _out(ea * zu.abs() + a.abs() * eu + 2 * U * h.abs(), h, bf16))}
    if dh is None:
        return out
    if bf16:                       # the kept pre-activations are rounded
        eg, eu = eg + BF * zg.abs(), eu + BF * zu.abs()
    G = dh.double()
    # act' is a sum of terms up to 1 + |z| times act'-like factors
    ea = D[gate] * eg + (16 + 4 * zg.abs()) * U * a.abs()
    ed = D2[gate] * eg + (16 + 4 * zg.abs()) * U * (1 + zg.abs() * torch.exp(-zg.abs() / 2))
    dg, du = G * zu * d, G * a
    dz = torch.cat((dg, du), 1)
    e = torch.cat((G.abs() * (eu * d.abs() + zu.abs() * ed) + 3 * U * dg.abs(), G.abs() * ea + 2 * U * du.abs()), 1)
    M = x.shape[0]
    db = dz.sum(0)
    out["db"] = (db, _out(e.sum(0) + 2 * M * U * dz.abs().sum(0), db, bf16))
    if bf16:
        e = e + BF * dz.abs()      # an operand of the two products
    dx, dw = dz @ W, dz.T @ X
    out["dx"] = (dx, _out(e @ W.abs() + 2 * 2 * F * U * (dz.abs() @ W.abs()), dx, bf16))
    out["dw"] = (dw, _out(e.T @ X.abs() + 2 * M * U * (dz.abs().T @ X.abs()), dw, bf16))
    return out


def adapter(x, w, a, b, ids, scale, bias, dy=None):
    """{name: (reference, bound)} of Y (and dX, dA, dB with dy); CPU tensors of one type."""
    bf16 = x.dtype == torch.bfloat16
    split = 2.0 ** -16 if bf16 else 0.0        # the low-rank activations in two bfloat16 parts
    X, W, A, B = x.double(), w.double(), a.double(), b.double()
    n, r, K = a.shape
    N, M = w.shape[0], x.shape[0]
    sc = torch.ones(n, dtype=torch.float64) if scale is None else scale.double()
    y = X @ W.T
    e = 2 * K * U * (X.abs() @ W.abs().T)
    if bias is not None:
        y = y + bias.double()
        e = e + U * y.abs()
    rows = {i: torch.nonzero(ids == i).squeeze(1) for i in range(n)}
    S, eS = torch.zeros(M, r, dtype=torch.float64), torch.zeros(M, r, dtype=torch.float64)
    for i, t in rows.items():
        S[t] = sc[i] * (X[t] @ A[i].T)
        eS[t] = sc[i].abs() * 2 * (K + 1) * U * (X[t].abs() @ A[i].abs().T)
        low, mag = S[t] @ B[i].T, S[t].abs() @ B[i].abs().T
        y[t] += low
        e[t] += eS[t] @ B[i].abs().T + (2 * (r + 2) * U + split) * mag + 2 * U * (y[t].abs() + low.abs())
    out = {"y": (y, _out(e, y, bf16))}
    if dy is None:
        return out
    G = dy.double()
    dx = G @ W
    e = 2 * N * U * (G.abs() @ W.abs())
    dA, eA, dB, eB = (torch.zeros_like(v) for v in (A, A, B, B))
    for i, t in rows.items():
        P = sc[i] * (G[t] @ B[i])
        eP = sc[i].abs() * 2 * (N + 1) * U * (G[t].abs() @ B[i].abs())
        low, mag = P @ A[i], P.abs() @ A[i].abs()
        dx[t] += low
        e[t] += eP @ A[i].abs() + (2 * (r + 2) * U + split) * mag + 2 * U * (dx[t].abs() + low.abs())
        T = len(t)
        dA[i], dB[i] = P.T @ X[t], G[t].T @ S[t]
        eA[i] = eP.T @ X[t].abs() + (2 * T * U + split) * (P.abs().T @ X[t].abs())
        eB[i] = G[t].abs().T @ eS[t] + (2 * T * U + split) * (G[t].abs().T @ S[t].abs())
    out["dx"] = (dx, _out(e, dx, bf16))
    out["da"] = (dA, _out(eA, dA, bf16))
    out["db"] = (dB, _out(eB, dB, bf16))
    return out


def check(got, ref_bound, label):
    """Assert |got - reference| <= bound element by element; the worst ratio."""
    ref, bound = ref_bound
    assert got.shape == ref.shape, f"{label}: shape {tuple(got.shape)}, expected {tuple(ref.shape)}"
    if ref.numel() == 0:
        return 0.0
    err = (got.double().cpu() - ref).abs()
    ratio = (err / bound).max().item()
    bad = ~(err <= bound)
    assert not bad.any(), (f"{label}: {int(bad.sum())} of {ref.numel()} elements exceed the bound, worst {ratio:.3g}x, "
                           f"first at {torch.nonzero(bad)[0].tolist()}")
    return ratio
