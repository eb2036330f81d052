"""64-bit definitions of the experts' operators and of products with 4-bit weights,
with the elementwise error bounds that the GPU tests hold the kernels to.

Bounds, derived from the arithmetic as in ops_reference (u = 2^-24):
  a product of K terms summed in FP32: 2 K u sum|a b|; from FP32 operands in three BF16
  parts the three smallest of nine products are left out: with 2^e <= |x| < 2^(e+1) the
  parts are |x1| <= 2^e <= |x| and |x2| <= 2^(e-1) <= |x| / 2 (8 bits to nearest leave
  half of the last), so 2^-24 (x1 w2 + x2 w1) is at most 2^-24 |x w| = u of a term;
  4-bit weights with few rows: each group of g columns sums (16 + q) x and (16 + zero) x,
  2 (g + 4) u of their magnitudes, scaled; the groups' sums 2 (G + 16) u more, G groups
  in eight waves' parts;
  with many rows the weight is rounded to the call's type before the product.
"""
import torch

import ops_reference as ref
from ops_reference import BF, D, D2, U, act64

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def order(ids, n):
    """offsets, pairs, places of ids [T, k], int32."""
    flat = ids.reshape(-1).tolist()
    rows = [[] for _ in range(n)]
    for p, e in enumerate(flat):
        if 0 <= e < n:
            rows[e].append(p)
    pairs = [p for r in rows for p in r]
    offsets = [0]
    for r in rows:
        offsets.append(offsets[-1] + len(r))
    places = [-1] * len(flat)
    for at, p in enumerate(pairs):
        places[p] = at
    pairs += [-1] * (len(flat) - len(pairs))
    return (torch.tensor(offsets, dtype=torch.int32), torch.tensor(pairs, dtype=torch.int32).reshape(-1),
            torch.tensor(places, dtype=torch.int32).reshape(ids.shape))


def make_ids(kind, T, k, n, seed=0):
    """ids [T, k]: 'mixed' (some outside [0, n)), 'one' (all of the last expert), 'none', 'few' (experts 1 and
    n - 1 alone), 'full' (every one inside)."""
    g = torch.Generator().manual_seed(seed)
    if kind == "one":
        return torch.full((T, k), n - 1, dtype=torch.int32)
    if kind == "none":
        return torch.where(torch.rand(T, k, generator=g) < 0.5, -1, n + 3).int()
    if kind == "few":
        return torch.where(torch.rand(T, k, generator=g) < 0.5, min(1, n - 1), n - 1).int()
    ids = torch.randint(0, max(n, 1), (T, k), generator=g)
    if kind == "mixed":
        bad = torch.tensor([-1, n, -(1 << 31), (1 << 31) - 1])[torch.randint(0, 4, (T, k), generator=g)]
        ids = torch.where(torch.rand(T, k, generator=g) < 0.2, bad, ids)
    return ids.int()


def combine(ys, places, weights, dy=None):
    """y (and dys, dw with dy)."""
    bf16 = ys.dtype == torch.bfloat16
    T, k = places.shape
    Y, w = ys.double(), torch.ones(T, k, dtype=torch.float64, device=ys.device) if weights is None else weights.double()
    there = (places >= 0).double()
    rows = Y[places.long().clamp(min=0).reshape(-1)].view(T, k, -1) if Y.shape[0] else Y.new_zeros(T, k, Y.shape[1])
    # rows of pairs that come nowhere may hold anything
    rows = torch.where(there.unsqueeze(2) > 0, rows, 0)
    y = (rows * (w * there).unsqueeze(2)).sum(1)
    mag = (rows.abs() * (w * there).abs().unsqueeze(2)).sum(1)
    out = {"y": (y, ref._out((k + 1) * U * mag, y, bf16))}
    if dy is None:
        return out
    G = dy.double()
    dys, e = torch.zeros_like(Y), torch.zeros_like(Y)
    for t in range(T):
        for j in range(k):
            if places[t, j] >= 0:
                dys[places[t, j]] = w[t, j] * G[t]
    dw = (rows * G.unsqueeze(1)).sum(2) * there
    mag = (rows.abs() * G.abs().unsqueeze(1)).sum(2)
    out["dys"] = (dys, ref._out(U * dys.abs() + e, dys, bf16))
    out["dw"] = (dw, ref._out(2 * (Y.shape[1] + 1) * U * mag, dw, False))
    return out


def _spans(offsets):
    o = offsets.tolist()
    return list(zip(o, o[1:]))


def _epilogue(z, ez, gate, bf16):
    """H, its bound and what the backward needs, from pre-activations and their bound."""
    if gate is None:
        return z, ref._out(ez, z, bf16), None
    F = z.shape[1] // 2
    zg, zu, eg, eu = z[:, :F], z[:, F:], ez[:, :F], ez[:, F:]
    a, d = act64(zg, gate)
    ea = D[gate] * eg + (16 + 4 * zg.abs()) * U * a.abs()
    h = a * zu
    return h, ref._out(ea * zu.abs() + a.abs() * eu + 2 * U * h.abs(), h, bf16), (a, d, ea, zg, zu, eg, eu)


def experts(x, w, offsets, bias, gate, dh=None):
    """{name: (reference, bound)} of H (and dx, dw, db with dh); CPU tensors of one type."""
    bf16 = x.dtype == torch.bfloat16
    left = 0.0 if bf16 else 1.0                       # products left out, in u of a term
    X, W = x.double(), w.double()
    n, N, K = w.shape
    P = x.shape[0]
    out_cols = N if gate is None else N // 2
    h, eh = torch.zeros(P, out_cols, dtype=torch.float64, device=x.device), torch.zeros(P, out_cols, dtype=torch.float64, device=x.device)
    dx, edx = torch.zeros_like(X), torch.zeros_like(X)
    dw, edw = torch.zeros_like(W), torch.zeros_like(W)
    db, edb = torch.zeros(n, N, dtype=torch.float64, device=x.device), torch.zeros(n, N, dtype=torch.float64, device=x.device)
    for e, (s, t) in enumerate(_spans(offsets)):
        if s == t:
            continue
        xe, R = X[s:t], t - s
        z = xe @ W[e].T
        ez = (2 * K + left) * U * (xe.abs() @ W[e].abs().T)
        if bias is not None:
            z = z + bias[e].double()
            ez = ez + U * z.abs()
        h[s:t], eh[s:t], kept = _epilogue(z, ez, gate, bf16)
        if dh is None:
            continue
        G = dh[s:t].double()
        if gate is None:
            dz, ed = G, torch.zeros_like(G)
        else:
            a, d, ea, zg, zu, eg, eu = kept
            ed = D2[gate] * eg + (16 + 4 * zg.abs()) * U * (1 + zg.abs() * torch.exp(-zg.abs() / 2))
            dg, du = G * zu * d, G * a
            dz = torch.cat((dg, du), 1)
            ed = torch.cat((G.abs() * (eu * d.abs() + zu.abs() * ed) + 3 * U * dg.abs(),
                            G.abs() * ea + 2 * U * du.abs()), 1)
        db[e] = dz.sum(0)
        edb[e] = ed.sum(0) + 2 * R * U * dz.abs().sum(0)
        if bf16 and gate is not None:
            ed = ed + BF * dz.abs()                   # an operand of the two products
        dx[s:t] = dz @ W[e]
        edx[s:t] = ed @ W[e].abs() + (2 * N + left) * U * (dz.abs() @ W[e].abs())
        dw[e] = dz.T @ xe
        edw[e] = ed.T @ xe.abs() + (2 * R + left) * U * (dz.abs().T @ xe.abs())
    out = {"h": (h, eh + ref.TINY)}
    if dh is not None:
        out["dx"], out["dw"], out["db"] = ((v, ref._out(b, v, bf16)) for v, b in ((dx, edx), (dw, edw), (db, edb)))
    return out


def weights4(q, scale, zero, group):
    """(q - zero) scale in 64 bits, and (32 + q + zero) scale, what the offset sums run over."""
    K = q.shape[-1]
    column = torch.arange(K) // group
    s = scale.double()[..., column]
    z = 8.0 if zero is None else zero.double()[..., column]
    return (q.double() - z) * s, (32 + q.double() + z) * s.abs()


def quant4(x, q, scale, zero, group, offsets, bias, gate, few):
    """(H, bound) for one bank [n, N, K] of 4-bit weights."""
    bf16 = x.dtype == torch.bfloat16
    w, mags = weights4(q, scale, zero, group)
    X = x.double()
    n, N, K = q.shape
    out_cols = N if gate is None else N // 2
    h, eh = torch.zeros(x.shape[0], out_cols, dtype=torch.float64, device=x.device), torch.zeros(x.shape[0], out_cols, dtype=torch.float64, device=x.device)
    for e, (s, t) in enumerate(_spans(offsets)):
        if s == t:
            continue
        xe = X[s:t]
        z, mag = xe @ w[e].T, xe.abs() @ w[e].abs().T
        if few:
            G = -(-K // group)
            ez = 2 * (group + 4) * U * (xe.abs() @ mags[e].T) + 2 * (G + 16) * U * mag
        else:
            ez = (2 * K + 2) * U * mag + (BF if bf16 else U) * mag
        if bias is not None:
            z = z + bias[e].double()
            ez = ez + U * z.abs()
        h[s:t], eh[s:t], _ = _epilogue(z, ez, gate, bf16)
    return h, eh + ref.TINY
