"""Feed-forward experts and layers with 4-bit weights: what they are measured on.

dispatch  tokens sorted by expert: the pairs (token, choice) of ids [T, k] in the
          order of their experts, stable; xs[r] = x[token of pair r].  Pairs whose id
          lies outside [0, n) come nowhere; xs is zero behind the last row.
combine   the way back: y[t] = sum over j of weights[t, j] ys[row of pair (t, j)]
experts   the experts' products on sorted rows: Z = xs_e W_e^T + bias_e for the rows
          of expert e, W [n, N, K]; with a gate H = act(Z[:, :F]) * Z[:, F:], N = 2F
q4        the same with weights of 4 bits, W = (q - zero) scale for each group of g
          columns of a row, of one layer or of experts

Each in the directions that it is used in: forward, and forward and backward
(`_train`).  `run` computes them in elementary torch operations in 32 bits, rounded
once at the end, or, where `own` is true, through the calls of this repository's
package.
"""
import math
import random

import torch

own = False

_DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def listed():
    return [
        # one token each of 16 requests, two experts each: latency
        {"name": "dispatch_f32_tokens", "op": "dispatch", "dtype": "f32", "T": 16, "k": 2, "n": 8, "K": 1024},
        # a training step's packed sequences over many experts, with the gradient of the tokens
        {"name": "dispatch_bf16_train", "op": "dispatch_train", "dtype": "bf16", "T": 16384, "k": 4, "n": 64,
         "K": 2048},
        # the small interatomic system (192 atoms, 32 tokens each): outputs, gradients of rows and weights
        {"name": "combine_f32_train", "op": "combine_train", "dtype": "f32", "T": 6144, "k": 2, "n": 16, "K": 256},
        # long prompts, eight experts a token, a width that no vector divides evenly
        {"name": "combine_bf16_prompts", "op": "combine", "dtype": "bf16", "T": 8191, "k": 8, "n": 64, "K": 2044},
        # one token each of 16 requests through the gated projection of 32 experts: the weights' bytes
        {"name": "experts_bf16_tokens", "op": "experts", "dtype": "bf16", "T": 16, "k": 2, "n": 32, "K": 2048,
         "N": 2816, "act": "silu", "bias": False},
        # long prompts through the experts' down projection: the matrix units' rate
        {"name": "experts_bf16_prompts", "op": "experts", "dtype": "bf16", "T": 16384, "k": 2, "n": 16, "K": 4096,
         "N": 2048, "act": None, "bias": False},
        # a training step of the interatomic block's width over eight experts, with bias gradients
        {"name": "experts_f32_train", "op": "experts_train", "dtype": "f32", "T": 6144, "k": 2, "n": 8, "K": 256,
         "N": 1024, "act": "gelu", "bias": True},
        # a training step on packed sequences (a row count and a hidden width that no tile divides)
        {"name": "experts_bf16_train", "op": "experts_train", "dtype": "bf16", "T": 8191, "k": 2, "n": 16, "K": 2048,
         "N": 2730, "act": "silu", "bias": False},
        # one token of one request through a wide layer: latency and the weights' bytes
        {"name": "q4_bf16_token", "op": "q4", "dtype": "bf16", "T": 1, "k": 0, "n": 1, "K": 4096, "N": 4096, "g": 128,
         "zero": True, "act": None, "bias": False},
        # one token each of 16 requests through a gated projection, float32 tensors, fine groups
        {"name": "q4_f32_tokens", "op": "q4", "dtype": "f32", "T": 16, "k": 0, "n": 1, "K": 1024, "N": 8192, "g": 32,
         "zero": True, "act": "silu", "bias": True},
        # one token each of 32 requests through the gated projections of 64 experts
        {"name": "q4_bf16_experts", "op": "q4", "dtype": "bf16", "T": 32, "k": 2, "n": 64, "K": 2048, "N": 2816,
         "g": 128, "zero": False, "act": "silu", "bias": False},
        # a prompt through a layer served in 4 bits
        {"name": "q4_bf16_prompt", "op": "q4", "dtype": "bf16", "T": 2047, "k": 0, "n": 1, "K": 4096, "N": 4096,
         "g": 64, "zero": True, "act": None, "bias": False},
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
    op = rng.choice(("dispatch", "dispatch_train", "combine", "combine_train", "experts", "experts", "experts_train",
                     "q4", "q4", "q4"))
    dtype = rng.choice(("f32", "bf16"))
    case = {"op": op, "dtype": dtype}
    if op.startswith(("dispatch", "combine")):
        # rows of tokens: bounded by the largest listed bytes
        case["n"] = _log(rng, 1, 128)
        case["k"] = rng.randint(1, min(8, case["n"]))
        case["K"] = _size(rng, 64, 4096)
        case["T"] = 1
        case["T"] = _size(rng, 1, max(1, int(min(16384, 5.0e8 / work(case)["bytes"]))))
        return case
    case["act"] = rng.choice((None, "silu", "gelu"))
    case["bias"] = rng.random() < 0.5
    case["K"], case["N"] = _size(rng, 64, 4096), 2 * _size(rng, 64, 2048)
    experts = op != "q4" or rng.random() < 0.5
    case["n"] = _log(rng, 1, 64) if experts else 1
    case["k"] = rng.randint(1, min(8, case["n"])) if experts else 0
    # a bank of at most the largest listed one's size
    case["n"] = max(1, min(case["n"], int((3.7e8 if op == "q4" else 1.4e8) / (case["K"] * case["N"]))))
    case["k"] = min(case["k"], case["n"])
    if op == "q4":
        case["g"], case["zero"] = rng.choice((32, 64, 128)), rng.random() < 0.5
    # rows: single tokens and prompts; a step trains on many rows; bounded by the largest listed work
    # of the type and the direction
    most = {("f32", False): 4.0e10, ("bf16", False): 4.0e11, ("f32", True): 4.0e10, ("bf16", True): 4.0e11}
    train = op.endswith("_train")
    per_pair = 2.0 * case["K"] * case["N"] * (3 if train else 1)
    hi = int(min(16384, most[dtype, train] / (per_pair * max(case["k"], 1))))
    if op == "q4" and rng.random() < 0.7:
        hi = min(hi, 64)
    case["T"] = _size(rng, min(64, max(1, hi)), max(1, hi)) if train else _size(rng, 1, max(1, hi))
    return case


def _choices(case, g, dev):
    """ids [T, k]: k different experts a token, some experts liked more than others; about one token in
    32 is padding and has none (-1)."""
    T, k, n = case["T"], case["k"], case["n"]
    liking = torch.randn((n,), generator=g, device=dev) * 0.5
    scores = torch.randn((T, n), generator=g, device=dev) + liking
    ids = scores.topk(k, dim=1).indices.to(torch.int32)
    padding = torch.rand((T, 1), generator=g, device=dev) < 1 / 32
    return torch.where(padding, -1, ids).contiguous()


def _sorted(ids, n):
    """offsets [n + 1], pairs [T k] (-1 behind the last), rows [T, k] (-1: none) of the pairs in the
    order of their experts."""
    flat = ids.reshape(-1).long()
    key = torch.where((flat >= 0) & (flat < n), flat, n)
    key, pairs = torch.sort(key, stable=True)
    offsets = (key.unsqueeze(0) < torch.arange(n + 1, device=ids.device).unsqueeze(1)).sum(dim=1)
    places = torch.empty_like(pairs)
    places[pairs] = torch.arange(pairs.numel(), device=ids.device)
    places = torch.where(places < offsets[n], places, -1)
    pairs = torch.where(key < n, pairs, -1)
    return offsets.to(torch.int32), pairs.to(torch.int32), places.to(torch.int32).view(ids.shape)


def _inputs(case, seed):
    """Tensors of the case on the GPU, in its type."""
    dt, dev = _DTYPES[case["dtype"]], torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)

    def normal(shape, sigma=1.0):
        return (torch.randn(shape, generator=g, device=dev, dtype=torch.float32) * sigma).to(dt)

    op, T, k, n, K = case["op"], case["T"], case["k"], case["n"], case["K"]
    t = {}
    P = T * max(k, 1)
    if k > 0:
        t["ids"] = _choices(case, g, dev)
        t["offsets"], t["pairs"], t["places"] = _sorted(t["ids"], n)
        rows = t["offsets"].tolist()
    else:
        rows = [0, T]
    if op.startswith("dispatch"):
        t["x"] = normal((T, K))
        if op == "dispatch_train":
            t["dxs"] = normal((P, K))
        return t
    if op.startswith("combine"):
        t["ys"] = normal((P, K))
        t["weights"] = torch.softmax(torch.randn((T, k), generator=g, device=dev), dim=1)
        if op == "combine_train":
            t["dy"] = normal((T, K))
        return t
    N = case["N"]
    t["spans"] = [(s, e) for s, e in zip(rows, rows[1:])]
    t["xs"] = normal((P, K))
    if k > 0:
        t["xs"][rows[-1]:] = 0                   # as the dispatch leaves them
    stacked = (n,) if k > 0 else ()              # one layer, or a bank of experts
    t["bias"] = normal(stacked + (N,), 0.1) if case["bias"] else None
    if op == "q4":
        groups = -(-K // case["g"])
        t["q"] = torch.randint(0, 16, stacked + (N, K), generator=g, device=dev, dtype=torch.uint8)
        # values of a spread of about K ** -0.5, as a weight of that spread is held
        t["scale"] = (torch.rand(stacked + (N, groups), generator=g, device=dev) + 0.5) * (0.22 * K ** -0.5)
        t["zero"] = None
        if case["zero"]:
            t["zero"] = torch.randint(6, 10, stacked + (N, groups), generator=g, device=dev, dtype=torch.uint8)
        return t
    t["w"] = normal((n, N, K), K ** -0.5)
    if op == "experts_train":
        t["dh"] = normal((P, N // 2 if case["act"] else N))
    return t


def prepare(case, seed):
    t = _inputs(case, seed)
    t["case"] = dict(case)
    if own:
        # what a program keeps: the order of this step's tokens, packed weights, leaves that require gradients
        from fp32_emulated_gemm_amd import experts, quant4
        op = case["op"]
        t["order"] = None
        if case["k"] > 0 and not op.startswith("dispatch"):
            t["order"] = experts.sort_tokens(t["ids"], case["n"])
        if op == "q4":
            t["packed"] = quant4.pack(t["q"], t["scale"], t["zero"], group=case["g"])
        leaves = {"dispatch_train": ("x",), "combine_train": ("ys", "weights"), "experts_train": ("xs", "w", "bias")}
        for name in leaves.get(op, ()):
            if t[name] is not None:
                t[name].requires_grad_(True)
    return t


# ---------------------------------------------------------------- the package's calls

def _run_own(t):
    from fp32_emulated_gemm_amd.experts import combine_tokens, expert_linear, gather_tokens, sort_tokens
    from fp32_emulated_gemm_amd.quant4 import quant4_linear
    case = t["case"]
    op = case["op"]
    if op.startswith("dispatch"):
        order = sort_tokens(t["ids"], case["n"])
        xs = gather_tokens(t["x"], order)
        out = [order.offsets, order.pairs, order.places, xs.detach()]
        return out + list(torch.autograd.grad(xs, (t["x"],), t["dxs"])) if op == "dispatch_train" else out
    if op.startswith("combine"):
        y = combine_tokens(t["ys"], t["order"], t["weights"])
        if op == "combine":
            return [y]
        return [y.detach(), *torch.autograd.grad(y, (t["ys"], t["weights"]), t["dy"])]
    if op == "q4":
        return [quant4_linear(t["xs"], t["packed"], bias=t["bias"], gate=case["act"], order=t["order"])]
    h = expert_linear(t["xs"], t["w"], t["order"], bias=t["bias"], gate=case["act"])
    if op == "experts":
        return [h]
    leaves = [t[name] for name in ("xs", "w", "bias") if t[name] is not None]
    return [h.detach(), *torch.autograd.grad(h, leaves, t["dh"])]


# ---------------------------------------------------------------- the plain forms

def _act(g, kind):
    """act(g) and its derivative, float32."""
    if kind == "silu":
        s = torch.sigmoid(g)
        return g * s, s * (1 + g * (1 - s))
    cdf = 0.5 * torch.special.erfc(g * -math.sqrt(0.5))
    return g * cdf, cdf + g * torch.exp(-0.5 * g * g) * (2 * math.pi) ** -0.5


def _plain_dispatch(t, train):
    case, dt = t["case"], t["x"].dtype
    offsets, pairs, places = _sorted(t["ids"], case["n"])
    token = pairs.long().clamp(min=0) // case["k"]
    out = [offsets, pairs, places, torch.where((pairs >= 0).unsqueeze(1), t["x"][token], 0)]
    if train:
        dxs = t["dxs"].float()
        dx = torch.zeros(t["x"].shape, dtype=torch.float32, device=dxs.device)
        for j in range(case["k"]):
            row = places[:, j].long()
            dx += torch.where((row >= 0).unsqueeze(1), dxs[row.clamp(min=0)], 0)
        out.append(dx.to(dt))
    return out


def _plain_combine(t, train):
    case, dt, weights = t["case"], t["ys"].dtype, t["weights"]
    ys, places = t["ys"].float(), t["places"].long()
    T = case["T"]
    y = torch.zeros((T, case["K"]), dtype=torch.float32, device=ys.device)
    for j in range(case["k"]):
        row = places[:, j]
        y += torch.where((row >= 0).unsqueeze(1), ys[row.clamp(min=0)] * weights[:, j:j + 1], 0)
    if not train:
        return [y.to(dt)]
    dy = t["dy"].float()
    pair = t["pairs"].long()
    there = (pair >= 0).unsqueeze(1)
    pair = pair.clamp(min=0)
    mine = dy[pair // case["k"]]
    dys = torch.where(there, mine * weights.reshape(-1)[pair].unsqueeze(1), 0)
    dot = (mine * ys).sum(dim=1)
    dw = torch.where(places >= 0, dot[places.clamp(min=0)], 0)
    return [y.to(dt), dys.to(dt), dw]


def _plain_weight(t, e):
    """Expert e's weight (or the layer's) in 32 bits."""
    case = t["case"]
    if case["op"] != "q4":
        return t["w"][e].float()
    q, scale = (t["q"][e], t["scale"][e]) if case["k"] > 0 else (t["q"], t["scale"])
    zero = 8.0
    if t["zero"] is not None:
        zero = (t["zero"][e] if case["k"] > 0 else t["zero"]).float()
        zero = zero.repeat_interleave(case["g"], dim=1)[:, :case["K"]]
    return (q.float() - zero) * scale.repeat_interleave(case["g"], dim=1)[:, :case["K"]]


def _plain_experts(t, train):
    case, dt = t["case"], t["xs"].dtype
    x = t["xs"].float()
    F = case["N"] // 2 if case["act"] else case["N"]
    h = torch.zeros((x.shape[0], F), dtype=torch.float32, device=x.device)
    if train:
        dh, dx, dw = t["dh"].float(), torch.zeros_like(x), torch.zeros(t["w"].shape, device=x.device)
        db = torch.zeros(t["bias"].shape, device=x.device) if case["bias"] else None
    for e, (s, stop) in enumerate(t["spans"]):
        if s == stop:
            continue
        w = _plain_weight(t, e)
        z = x[s:stop] @ w.t()
        if case["bias"]:
            z += (t["bias"][e] if case["k"] > 0 else t["bias"]).float()
        if case["act"]:
            act, dact = _act(z[:, :F], case["act"])
            h[s:stop] = act * z[:, F:]
        else:
            h[s:stop] = z
        if train:
            dz = dh[s:stop]
            if case["act"]:
                dz = torch.cat((dz * z[:, F:] * dact, dz * act), dim=1)
            dx[s:stop] = dz @ w
            dw[e] = dz.t() @ x[s:stop]
            if case["bias"]:
                db[e] = dz.sum(dim=0)
    if not train:
        return [h.to(dt)]
    out = [h.to(dt), dx.to(dt), dw.to(dt)]
    return out + [db.to(dt)] if case["bias"] else out


def run(state):
    if own:
        return _run_own(state)
    op = state["case"]["op"]
    train = op.endswith("_train")
    if op.startswith("dispatch"):
        return _plain_dispatch(state, train)
    if op.startswith("combine"):
        return _plain_combine(state, train)
    return _plain_experts(state, train)


# ---------------------------------------------------------------- cost and the 64-bit definition

def work(case):
    size = 4 if case["dtype"] == "f32" else 2
    op, T, K = case["op"], case["T"], case["K"]
    P = T * max(case["k"], 1)
    if op.startswith("dispatch"):
        moved = size * K * (T + P) + 4 * (3 * P + case["n"] + 1)       # ids, pairs, places; x, xs
        if op == "dispatch":
            return {"bytes": moved, "flops": 0.0}
        return {"bytes": moved + size * K * (T + P), "flops": 1.0 * P * K}
    if op.startswith("combine"):
        moved = size * K * (T + P) + 8 * P                              # ys, y; places, weights
        if op == "combine":
            return {"bytes": moved, "flops": 2.0 * P * K}
        # dy read, dys and the weights' gradients written
        return {"bytes": moved + size * K * (T + P) + 8 * P, "flops": 5.0 * P * K}
    N, n = case["N"], case["n"]
    F = N // 2 if case["act"] else N
    used = max(1, int(n * (1 - (1 - 1 / n) ** P))) if n > 1 else 1       # experts that have rows, about
    bias = size * N if case["bias"] else 0
    if op == "q4":
        groups = -(-K // case["g"])
        weights = used * N * (K / 2 + groups * (5 if case["zero"] else 4))
    else:
        weights = used * N * K * size
    flops = 2.0 * P * K * N
    forward = size * P * (K + F) + weights + used * bias
    if op != "experts_train":
        return {"bytes": forward, "flops": flops}
    # dh read, dx, dw and db written
    return {"bytes": forward + size * P * (K + F) + size * n * N * K + n * bias, "flops": 3 * flops}


def exact(case, seed):
    """The definitions in float64, pair by pair or expert by expert."""
    t = _inputs(case, seed)
    op, T, k, n, K = case["op"], case["T"], case["k"], case["n"], case["K"]
    train = op.endswith("_train")
    if op.startswith("dispatch"):
        ids = t["ids"].reshape(-1)
        lists = [torch.nonzero(ids == e).squeeze(1) for e in range(n)]      # ascending pairs of each expert
        pairs = torch.cat(lists)
        xs = torch.zeros((T * k, K), dtype=torch.float64, device=ids.device)
        xs[:pairs.numel()] = t["x"].double()[torch.div(pairs, k, rounding_mode="floor")]
        out = [None, None, None, xs]
        if train:
            dx = torch.zeros((T * k, K), dtype=torch.float64, device=ids.device)
            dx[pairs] = t["dxs"].double()[:pairs.numel()]
            out.append(dx.view(T, k, K).sum(dim=1))
        return out
    if op.startswith("combine"):
        ids = t["ids"].reshape(-1)
        pairs = torch.cat([torch.nonzero(ids == e).squeeze(1) for e in range(n)])
        m, w = pairs.numel(), t["weights"].double().reshape(-1)
        ys = t["ys"].double()
        parts = torch.zeros((T * k, K), dtype=torch.float64, device=ids.device)
        parts[pairs] = ys[:m] * w[pairs].unsqueeze(1)
        y = parts.view(T, k, K).sum(dim=1)
        if not train:
            return [y]
        back = t["dy"].double()[torch.div(pairs, k, rounding_mode="floor")]
        dys, dw = torch.zeros_like(ys), torch.zeros_like(w)
        dys[:m] = back * w[pairs].unsqueeze(1)
        dw[pairs] = (back * ys[:m]).sum(dim=1)
        return [y, dys, dw.view(T, k)]
    x = t["xs"].double()
    N = case["N"]
    F = N // 2 if case["act"] else N
    h = torch.zeros((x.shape[0], F), dtype=torch.float64, device=x.device)
    dx, grads = torch.zeros_like(x), []
    for e, (s, stop) in enumerate(t["spans"]):
        bank = (lambda v: v[e]) if k > 0 else (lambda v: v)
        if op == "q4":
            column = torch.arange(K, device=x.device) // case["g"]
            zero = 8 if t["zero"] is None else bank(t["zero"]).double()[:, column]
            w = (bank(t["q"]).double() - zero) * bank(t["scale"]).double()[:, column]
        else:
            w = t["w"][e].double()
        z = x[s:stop] @ w.T.contiguous()
        if case["bias"]:
            z = z + bank(t["bias"]).double()
        dz = t["dh"][s:stop].double() if train else None
        if case["act"]:
            a, u = z[:, :F], z[:, F:]
            if case["act"] == "silu":
                gate = 1 / (1 + torch.exp(-a))
                slope = gate + a * gate * (1 - gate)
            else:
                gate = torch.special.ndtr(a)
                slope = gate + a * torch.exp(-a * a / 2) / math.sqrt(2 * math.pi)
            h[s:stop] = a * gate * u
            if train:
                dz = torch.cat((dz * u * slope, dz * a * gate), dim=1)
        else:
            h[s:stop] = z
        if train:
            dx[s:stop] = dz @ w
            grads.append((dz.T.contiguous() @ x[s:stop], dz.sum(dim=0)))
    if not train:
        return [h]
    out = [h, dx, torch.stack([dw for dw, _ in grads])]
    return out + [torch.stack([db for _, db in grads])] if case["bias"] else out
