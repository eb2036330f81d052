"""The gated feed-forward projection and the linear layer with low-rank adapters:
what they are measured on.

Two operators, each forward (for prompts and for single tokens) and as a training
step (forward and backward), for float32 and bfloat16 tensors:

gated     H = act(Z[:, :F]) * Z[:, F:],  Z = X W^T + bias,  W [2F, K]: the gate's
          rows, then the up projection's
adapter   Y[t] = W X[t] + bias + scale[i] B[i] (A[i] X[t]),  i = ids[t];
          A [n, r, K], B [n, N, r]; a row whose id is negative has no adapter

`run` computes them in elementary torch operations in 32 bits, rounded once at
the end, or, where `own` is true, through the calls of this repository's package.
"""
import math
import random

import torch

own = False

_DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def listed():
    return [
        # one token of one request through a feed-forward block: latency and the weights' bytes
        {"name": "gated_f32_token", "op": "gated", "dtype": "f32", "M": 1, "K": 1024, "F": 4096,
         "act": "silu", "bias": False},
        # the feed-forward block of the small interatomic system: 192 atoms, 32 tokens each
        {"name": "gated_f32_small_box", "op": "gated", "dtype": "f32", "M": 6144, "K": 256, "F": 1024,
         "act": "gelu", "bias": True},
        # one token each of 48 requests served together
        {"name": "gated_bf16_tokens", "op": "gated", "dtype": "bf16", "M": 48, "K": 4096, "F": 8192,
         "act": "silu", "bias": False},
        # a long prompt batch through a wide block: the matrix units' rate
        {"name": "gated_bf16_prompts", "op": "gated", "dtype": "bf16", "M": 8192, "K": 4096, "F": 8192,
         "act": "silu", "bias": False},
        # a training step of the interatomic block's width, with bias gradients
        {"name": "gated_f32_train", "op": "gated_train", "dtype": "f32", "M": 24576, "K": 256, "F": 1024,
         "act": "gelu", "bias": True},
        # a training step on packed sequences (a row count and a hidden width that no tile divides)
        {"name": "gated_bf16_train", "op": "gated_train", "dtype": "bf16", "M": 8191, "K": 2048, "F": 5461,
         "act": "silu", "bias": False},
        # one token each of 16 requests, each with its own adapter
        {"name": "adapter_f32_tokens", "op": "adapter", "dtype": "f32", "M": 16, "K": 1024, "N": 1024,
         "n": 32, "r": 8, "requests": 16, "bias": True},
        # one token each of 64 requests over a bank of 64 adapters
        {"name": "adapter_bf16_tokens", "op": "adapter", "dtype": "bf16", "M": 64, "K": 4096, "N": 4096,
         "n": 64, "r": 16, "requests": 64, "bias": False},
        # prompts of 11 requests, ragged lengths, some without an adapter
        {"name": "adapter_f32_prompts", "op": "adapter", "dtype": "f32", "M": 2111, "K": 1024, "N": 1024,
         "n": 8, "r": 16, "requests": 11, "bias": True},
        # long prompts of 24 requests, a high rank
        {"name": "adapter_bf16_prompts", "op": "adapter", "dtype": "bf16", "M": 8192, "K": 4096, "N": 4096,
         "n": 16, "r": 64, "requests": 24, "bias": False},
        # fine-tuning four adapters beside a fixed layer of the small interatomic system
        {"name": "adapter_f32_train", "op": "adapter_train", "dtype": "f32", "M": 6144, "K": 256, "N": 1024,
         "n": 4, "r": 8, "requests": 24, "bias": True},
        # fine-tuning eight adapters on packed sequences beside a wide fixed layer
        {"name": "adapter_bf16_train", "op": "adapter_train", "dtype": "bf16", "M": 8192, "K": 4096, "N": 4096,
         "n": 8, "r": 16, "requests": 16, "bias": False},
    ]


def _log(rng, lo, hi):
    """An integer spread evenly over the logarithm of [lo, hi]."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _size(rng, lo, hi):
    """A size in [lo, hi]: any integer one time in three, else a multiple of 64, 16 or 8."""
    v = _log(rng, lo, hi)
    step = rng.choice((1, 1, 8, 16, 64, 64))
    return max(lo, v - v % step)


def draw(rng: random.Random):
    op = rng.choice(("gated", "gated", "adapter", "adapter", "gated_train", "adapter_train"))
    dtype = rng.choice(("f32", "bf16"))
    train = op.endswith("_train")
    case = {"op": op, "dtype": dtype, "bias": rng.random() < 0.5}
    if op.startswith("gated"):
        case["K"], case["F"] = _size(rng, 192, 4096), _size(rng, 512, 8192)
        case["act"] = rng.choice(("silu", "gelu"))
    else:
        case["K"], case["N"] = _size(rng, 192, 4096), _size(rng, 192, 4096)
        case["n"], case["r"] = _log(rng, 1, 64), rng.choice((4, 8, 12, 16, 16, 32, 64))
    # rows: tokens and prompts; a step trains on 512 rows or more; bounded by the largest listed
    # work of the type and the direction
    most = {("f32", False): 4.0e10, ("bf16", False): 1.0e12, ("f32", True): 7.5e10, ("bf16", True): 8.0e11}
    case["M"] = 1
    if not op.startswith("gated"):
        case["requests"] = 1
    per_row = work(case)["flops"]
    hi = int(min(8192, most[dtype, train] / per_row))
    case["M"] = _size(rng, 512, max(512, hi)) if train else _size(rng, 1, max(1, hi))
    if not op.startswith("gated"):
        # single tokens, or requests of many rows each
        case["requests"] = case["M"] if case["M"] <= 64 and not train else rng.randint(1, min(32, case["M"]))
    return case


def _spans(M, requests, n, seed):
    """(first row, end, adapter) of each request; about one in eight has no adapter (-1)."""
    rng = random.Random(seed)
    cuts = sorted(rng.sample(range(1, M), requests - 1)) if requests > 1 else []
    edges = [0] + cuts + [M]
    return [(s, e, -1 if rng.random() < 0.125 else rng.randrange(n)) for s, e in zip(edges, edges[1:])]


def _inputs(case, seed):
    """Tensors of the case on the GPU, in its type, and the requests' row spans."""
    dt, dev = _DTYPES[case["dtype"]], torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)

    def normal(shape, sigma=1.0):
        return (torch.randn(shape, generator=g, device=dev, dtype=torch.float32) * sigma).to(dt)

    M, K = case["M"], case["K"]
    t = {"x": normal((M, K))}
    if case["op"].startswith("gated"):
        F = case["F"]
        t["w"] = normal((2 * F, K), K ** -0.5)
        t["bias"] = normal((2 * F,), 0.1) if case["bias"] else None
        if case["op"] == "gated_train":
            t["dh"] = normal((M, F))
        return t
    N, n, r = case["N"], case["n"], case["r"]
    t["w"] = normal((N, K), K ** -0.5)
    t["bias"] = normal((N,), 0.1) if case["bias"] else None
    t["a"], t["b"] = normal((n, r, K), K ** -0.5), normal((n, N, r), 0.5 * r ** -0.5)
    t["scale"] = torch.rand((n,), generator=g, device=dev, dtype=torch.float32) + 0.5
    t["spans"] = _spans(M, case["requests"], n, seed)
    rows = [i for s, e, i in t["spans"] for _ in range(e - s)]
    t["ids"] = torch.tensor(rows, dtype=torch.int32).to(dev)
    if case["op"] == "adapter_train":
        t["dy"] = normal((M, N))
    return t


def prepare(case, seed):
    t = _inputs(case, seed)
    t["case"] = dict(case)
    if own:
        # what a program keeps: the layouts of weights that do not change, and leaves that require gradients
        from fp32_emulated_gemm_amd import adapters, gated
        if case["op"] == "gated":
            t["plan"] = gated.plan_weight(t["w"])
        elif case["op"] == "gated_train":
            for name in ("x", "w", "bias"):
                if t[name] is not None:
                    t[name].requires_grad_(True)
        else:
            t["plan"] = adapters.plan_weight(t["w"], backward=case["op"] == "adapter_train")
            if case["op"] == "adapter_train":
                for name in ("x", "a", "b"):
                    t[name].requires_grad_(True)
    return t


# ---------------------------------------------------------------- the package's calls

def _run_own(t):
    from fp32_emulated_gemm_amd.adapters import adapter_linear
    from fp32_emulated_gemm_amd.gated import gated_linear
    case = t["case"]
    if case["op"] == "gated":
        return [gated_linear(t["x"], t["w"], t["bias"], gate=case["act"], plan=t["plan"])]
    if case["op"] == "gated_train":
        h = gated_linear(t["x"], t["w"], t["bias"], gate=case["act"])
        leaves = [t[name] for name in ("x", "w", "bias") if t[name] is not None]
        return [h.detach(), *torch.autograd.grad(h, leaves, t["dh"])]
    y = adapter_linear(t["x"], t["w"], t["a"], t["b"], t["ids"], scale=t["scale"], bias=t["bias"], plan=t["plan"])
    if case["op"] == "adapter":
        return [y]
    return [y.detach(), *torch.autograd.grad(y, (t["x"], t["a"], t["b"]), t["dy"])]


# ---------------------------------------------------------------- the plain forms

def _act(g, kind):
    """act(g) and its derivative, float32."""
    if kind == "silu":
        s = torch.sigmoid(g)
        return g * s, s * (1 + g * (1 - s))
    cdf = 0.5 * torch.special.erfc(g * -math.sqrt(0.5))
    return g * cdf, cdf + g * torch.exp(-0.5 * g * g) * (2 * math.pi) ** -0.5


def _plain_gated(t, train):
    dt, F = t["x"].dtype, t["case"]["F"]
    x, w = t["x"].float(), t["w"].float()
    z = x @ w.t()
    if t["bias"] is not None:
        z += t["bias"].float()
    act, dact = _act(z[:, :F], t["case"]["act"])
    h = (act * z[:, F:]).to(dt)
    if not train:
        return [h]
    dh = t["dh"].float()
    dz = torch.cat((dh * z[:, F:] * dact, dh * act), dim=1)
    out = [h, (dz @ w).to(dt), (dz.t() @ x).to(dt)]
    if t["bias"] is not None:
        out.append(dz.sum(dim=0).to(dt))
    return out


def _plain_adapter(t, train):
    dt = t["x"].dtype
    x, w, a, b, scale = t["x"].float(), t["w"].float(), t["a"].float(), t["b"].float(), t["scale"]
    y = x @ w.t()
    if t["bias"] is not None:
        y += t["bias"].float()
    if all(e - s == 1 for s, e, _ in t["spans"]):
        # single tokens: every row gathers its adapter
        i = t["ids"].long()
        k = i.clamp(min=0)
        low = torch.bmm(a[k], x.unsqueeze(2)) * (scale[k] * (i >= 0)).view(-1, 1, 1)
        y += torch.bmm(b[k], low).squeeze(2)
        return [y.to(dt)]
    lows = []
    for s, e, i in t["spans"]:
        low = None
        if i >= 0:
            low = (x[s:e] @ a[i].t()) * scale[i]
            y[s:e] += low @ b[i].t()
        lows.append(low)
    if not train:
        return [y.to(dt)]
    dy = t["dy"].float()
    dx = dy @ w
    da, db = torch.zeros_like(a), torch.zeros_like(b)
    for (s, e, i), low in zip(t["spans"], lows):
        if i >= 0:
            dlow = (dy[s:e] @ b[i]) * scale[i]
            dx[s:e] += dlow @ a[i]
            da[i] += dlow.t() @ x[s:e]
            db[i] += dy[s:e].t() @ low
    return [y.to(dt), dx.to(dt), da.to(dt), db.to(dt)]


def run(state):
    if own:
        return _run_own(state)
    op = state["case"]["op"]
    if op.startswith("gated"):
        return _plain_gated(state, op == "gated_train")
    return _plain_adapter(state, op == "adapter_train")


# ---------------------------------------------------------------- cost and the 64-bit definition

def work(case):
    size = 4 if case["dtype"] == "f32" else 2
    M, K = case["M"], case["K"]
    if case["op"].startswith("gated"):
        F = case["F"]
        flops = 2.0 * M * K * 2 * F
        weights = 2 * F * K + (2 * F if case["bias"] else 0)
        if case["op"] == "gated":
            return {"bytes": size * (M * K + weights + M * F), "flops": flops}
        # x, dh, w read; h, dx, dw written
        return {"bytes": size * (2 * M * K + 2 * weights + 2 * M * F), "flops": 3 * flops}
    N, n, r = case["N"], min(case["n"], case["requests"]), case["r"]
    base, low = 2.0 * M * N * K, 2.0 * M * r * (K + N)
    fixed, bank = N * K + (N if case["bias"] else 0), n * r * (K + N)
    if case["op"] == "adapter":
        return {"bytes": size * (M * K + fixed + bank + M * N) + 4 * M, "flops": base + low}
    # x, dy, w, a, b read; y, dx, da, db written
    return {"bytes": size * (2 * M * K + fixed + 2 * bank + 2 * M * N) + 4 * M, "flops": 2 * base + 3 * low}


def exact(case, seed):
    """The definition in float64, row by adapter row."""
    t = _inputs(case, seed)
    x, w = t["x"].double(), t["w"].double()
    train = case["op"].endswith("_train")
    z = torch.matmul(x, w.T.contiguous())
    if t["bias"] is not None:
        z = z + t["bias"].double()
    if case["op"].startswith("gated"):
        g, u = z[:, :case["F"]], z[:, case["F"]:]
        if case["act"] == "silu":
            gate = 1 / (1 + torch.exp(-g))
            slope = gate + g * gate * (1 - gate)
        else:
            gate = torch.special.ndtr(g)
            slope = gate + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
        h = g * gate * u
        if not train:
            return [h]
        dh = t["dh"].double()
        dg, du = dh * u * slope, dh * g * gate
        F = case["F"]
        out = [h, dg @ w[:F] + du @ w[F:], torch.cat((dg.T.contiguous() @ x, du.T.contiguous() @ x))]
        if t["bias"] is not None:
            out.append(torch.cat((dg.sum(0), du.sum(0))))
        return out
    a, b, scale, ids = t["a"].double(), t["b"].double(), t["scale"].double(), t["ids"].long()
    dy = t["dy"].double() if train else None
    dx = dy @ w if train else None
    da, db = torch.zeros_like(a), torch.zeros_like(b)
    for i in sorted(set(ids.tolist()) - {-1}):
        rows = torch.nonzero(ids == i).squeeze(1)
        xi, delta = x[rows], scale[i] * (b[i] @ a[i])           # the adapter as a full matrix [N, K]
        z[rows] += xi @ delta.T.contiguous()
        if train:
            di = dy[rows]
            dx[rows] += di @ delta
            full = scale[i] * (di.T.contiguous() @ xi)           # the full matrix's gradient
            da[i] = b[i].T.contiguous() @ full
            db[i] = full @ a[i].T.contiguous()
    return [z, dx, da, db] if train else [z]
