"""Feed-forward experts: tokens sorted by expert and back, and the experts'
products, for float32 and bfloat16 tensors, with gradients:

    order = sort_tokens(ids, n)                 # ids [T, k]: each token's k experts
    xs = gather_tokens(x, order)                # [T k, K], rows in the order of their experts
    h = expert_linear(xs, w, order, gate="silu")    # w [n, 2F, K]: the gated projection of each row's expert
    ys = expert_linear(h, v, order)             # v [n, K, F]
    y = combine_tokens(ys, order, weights)      # y[t] = sum over j of weights[t, j] ys[row of (t, j)]

Nothing waits for the host: which rows belong to which expert stays on the device
(`order.offsets`), and rows of no expert (ids outside [0, n), as of padded tokens)
lie behind the last and are zeros.  All calls can be captured into graphs.
Gradients are deterministic.  The calls are those of include/sgemm_emu_experts.h.
"""
import ctypes

import torch

from .ops import (DTYPES, GATES, addr, check_tensor, forward_mode, ok, ops_lib, rows_of, scratch, stream_of)

SGEMM_EMU_MAX_EXPERTS = 1024
SGEMM_EMU_GATE_NONE = -1
SORT_IN_ONE = 1024   # pairs that the sort takes without workspace, at least: those calls need not ask

EXPERTS_EXPORTS = ("sgemm_emu_sort_tokens_workspace", "sgemm_emu_sort_tokens", "sgemm_emu_gather_tokens",
                   "sgemm_emu_combine_tokens", "sgemm_emu_combine_tokens_backward", "sgemm_emu_expert_linear",
                   "sgemm_emu_expert_linear_backward_workspace", "sgemm_emu_expert_linear_backward",
                   "sgemm_emu_quant4_bytes", "sgemm_emu_quant4_quantize", "sgemm_emu_quant4_pack",
                   "sgemm_emu_quant4_unpack", "sgemm_emu_quant4_linear_workspace", "sgemm_emu_quant4_linear")

_LIB = None


def experts_lib():
    """The library with these operators' signatures set (once)."""
    global _LIB
    if _LIB is None:
        L = ops_lib()
        i64, vp, ci = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int
        L.sgemm_emu_sort_tokens_workspace.argtypes = [i64, i64]
        L.sgemm_emu_sort_tokens.argtypes = [i64, i64, vp, vp, vp, vp, vp, i64, vp]
        L.sgemm_emu_gather_tokens.argtypes = [ci, i64, i64, i64, i64, vp, i64, vp, vp, vp, i64, vp]
        L.sgemm_emu_combine_tokens.argtypes = [ci, i64, i64, i64, vp, i64, vp, vp, vp, i64, vp]
        L.sgemm_emu_combine_tokens_backward.argtypes = [ci, i64, i64, i64, i64, vp, i64, vp, vp, vp, vp, i64, vp, i64,
                                                        vp, vp]
        bank = [ci, i64, i64, i64, i64]
        L.sgemm_emu_expert_linear.argtypes = bank + [vp, i64, vp, vp, ci, vp, vp, i64, vp, vp]
        L.sgemm_emu_expert_linear_backward_workspace.argtypes = bank + [ci, ci]
        L.sgemm_emu_expert_linear_backward.argtypes = bank + [vp, i64, vp, vp, ci, vp, vp, i64, vp, i64, vp, vp, vp,
                                                              i64, vp]
        L.sgemm_emu_quant4_bytes.argtypes = [i64, i64, i64, i64, ci]
        L.sgemm_emu_quant4_quantize.argtypes = bank + [vp, vp, vp, vp, vp]
        L.sgemm_emu_quant4_pack.argtypes = [i64, i64, i64, i64, vp, vp, vp, vp, vp]
        L.sgemm_emu_quant4_unpack.argtypes = bank + [ci, vp, vp, vp]
        L.sgemm_emu_quant4_linear_workspace.argtypes = bank + [i64, ci]
        L.sgemm_emu_quant4_linear.argtypes = bank + [i64, ci, vp, i64, vp, vp, ci, vp, vp, i64, vp, i64, vp]
        for name in EXPERTS_EXPORTS:
            getattr(L, name).restype = i64 if name.endswith(("_workspace", "_bytes")) else ci
        _LIB = L
    return _LIB


def value_type(t, name):
    """The type of a tensor argument that the others share."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch tensor, got {type(t).__name__}")
    if t.dtype not in DTYPES:
        raise TypeError(f"{name}: expected dtype float32 or bfloat16, got {t.dtype}")
    return t.dtype


def _differentiable(*tensors):
    """Whether a call on these has to go through its autograd function."""
    return forward_mode() or (torch.is_grad_enabled() and any([t is not None and t.requires_grad for t in tensors]))


def once(backward):
    """torch's once_differentiable, whose own time a backward pass that records nothing is spared."""
    recorded = torch.autograd.function.once_differentiable(backward)

    def run(ctx, *grads):
        return (recorded if torch.is_grad_enabled() else backward)(ctx, *grads)
    return run


# ---------------------------------------------------------------- tokens

class ExpertOrder:
    """The pairs (token, choice) of ids [T, k] in the order of their experts, as sort_tokens made it:
    `offsets` [n + 1]: expert e's rows are [offsets[e], offsets[e + 1]); `pairs` [T k]: sorted row -> pair
    t k + j, -1 behind the last; `places` [T, k]: pair -> sorted row, -1 where it comes nowhere.  int32."""

    __slots__ = ("offsets", "pairs", "places", "experts", "tokens", "choices", "rows", "device_index")

    def __init__(self, offsets, pairs, places, experts):
        self.offsets, self.pairs, self.places, self.experts = offsets, pairs, places, experts
        self.tokens, self.choices = places.shape
        self.rows = self.tokens * self.choices
        self.device_index = offsets.get_device() if offsets.is_cuda else None


def check_order(order):
    if not isinstance(order, ExpertOrder):
        raise TypeError(f"order: expected an ExpertOrder (of sort_tokens), got {type(order).__name__}")
    if order.device_index is None or order.device_index != torch.cuda.current_device():
        raise ValueError(f"order: expected one on the current HIP device, got {order.offsets.device}")


def _fits(t, order, rows):
    """check_order and check_tensor of a tensor of `rows` rows in one expression, for the calls where the
    host's time counts."""
    try:
        return (t.dtype in DTYPES and t.dim() == 2 and t.shape[0] == rows
                and t.get_device() == order.device_index == torch.cuda.current_device())
    except (AttributeError, RuntimeError):       # RuntimeError: no device
        return False


def sort_tokens(ids, experts):
    """The order of ids [T, k] (or [T]), int32 on the current HIP device, among `experts` experts.  Pairs
    of one expert keep their order; an id outside [0, experts) comes nowhere."""
    if not isinstance(ids, torch.Tensor):
        raise TypeError(f"ids: expected a torch tensor, got {type(ids).__name__}")
    dims = ids.dim()
    if dims not in (1, 2):
        raise ValueError(f"ids: expected one or two dimensions, got {dims}")
    if ids.dtype is not torch.int32 or not ids.is_cuda or ids.get_device() != torch.cuda.current_device():
        check_tensor(ids, "ids", torch.int32, ids.shape)
    if not 0 <= experts <= SGEMM_EMU_MAX_EXPERTS:
        raise ValueError(f"experts: expected 0 to {SGEMM_EMU_MAX_EXPERTS}, got {experts}")
    L = experts_lib()
    ids = ids.contiguous()
    T, P = ids.shape[0], ids.numel()
    out = ids.new_empty(2 * P + experts + 1)
    offsets, pairs, places = out.split_with_sizes((experts + 1, P, P))
    nws = 0
    if P > SORT_IN_ONE:
        nws = ok(L.sgemm_emu_sort_tokens_workspace(P, experts), "sgemm_emu_sort_tokens_workspace")
    ws = scratch(nws, ids)
    at = out.data_ptr()
    ok(L.sgemm_emu_sort_tokens(P, experts, addr(ids), at, at + 4 * (experts + 1), at + 4 * (experts + 1 + P), addr(ws), nws,
                               stream_of(ids.get_device())), "sgemm_emu_sort_tokens")
    return ExpertOrder(offsets, pairs, places.view(T, ids.shape[1] if dims == 2 else 1), experts)


def _gather(x, order):
    L = experts_lib()
    x, xld = rows_of(x)
    T, K = x.shape
    xs = x.new_empty((order.rows, K))
    ok(L.sgemm_emu_gather_tokens(DTYPES[x.dtype], T, order.choices, K, order.experts, addr(x), xld,
                                 addr(order.offsets), addr(order.places), addr(xs), max(K, 1),
                                 stream_of(x.get_device())), "sgemm_emu_gather_tokens")
    return xs


def _combine(ys, order, weights):
    L = experts_lib()
    ys, yld = rows_of(ys)
    K = ys.shape[1]
    y = ys.new_empty((order.tokens, K))
    ok(L.sgemm_emu_combine_tokens(DTYPES[ys.dtype], order.tokens, order.choices, K, addr(ys), yld, addr(order.places),
                                  addr(weights), addr(y), max(K, 1), stream_of(ys.get_device())),
       "sgemm_emu_combine_tokens")
    return y


class _GatherFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, order):
        ctx.order = order
        return _gather(x, order)

    @staticmethod
    @once
    def backward(ctx, dxs):
        return _combine(dxs, ctx.order, None), None


class _CombineFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, ys, order, weights):
        ctx.order = order
        # rows are read by the weights' gradient alone
        ctx.save_for_backward(ys if ctx.needs_input_grad[2] else None, weights)
        return _combine(ys, order, weights)

    @staticmethod
    @once
    def backward(ctx, dy):
        (ys, weights), order = ctx.saved_tensors, ctx.order
        L = experts_lib()
        (ys, yld), (dy, dyld) = (None, 1) if ys is None else rows_of(ys), rows_of(dy)
        K = dy.shape[1]
        dys = dy.new_empty((order.rows, K)) if ctx.needs_input_grad[0] else None
        dw = None if ys is None else torch.empty_like(weights)
        ok(L.sgemm_emu_combine_tokens_backward(DTYPES[dy.dtype], order.tokens, order.choices, K, order.experts,
                                               addr(ys), yld, addr(order.offsets), addr(order.places), addr(weights),
                                               addr(dy), dyld, addr(dys), max(K, 1), addr(dw),
                                               stream_of(dy.get_device())), "sgemm_emu_combine_tokens_backward")
        return dys, None, dw


def gather_tokens(x, order):
    """Rows x[t] of x [T, K] (float32 or bfloat16) in the order of their experts: [T k, K], zeros behind the
    last.  Differentiable in x, in reverse mode."""
    if not _fits(x, order, getattr(order, "tokens", None)):
        check_order(order)
        check_tensor(x, "x", value_type(x, "x"), (order.tokens, None))
    return _GatherFn.apply(x, order) if _differentiable(x) else _gather(x, order)


def combine_tokens(ys, order, weights=None):
    """y[t] = sum over j of weights[t, j] ys[row of pair (t, j)] for ys [T k, K] (float32 or bfloat16), summed
    in 32 bits with j ascending; weights: float32 [T, k], or None (1).  Pairs that come nowhere add nothing.
    Differentiable in ys and weights, in reverse mode."""
    if not _fits(ys, order, getattr(order, "rows", None)):
        check_order(order)
        check_tensor(ys, "ys", value_type(ys, "ys"), (order.rows, None))
    if weights is not None:
        if not (_fits(weights, order, order.tokens) and weights.dtype is torch.float32 and weights.shape[1] == order.choices):
            check_tensor(weights, "weights", torch.float32, (order.tokens, order.choices))
        weights = weights.contiguous()
    return _CombineFn.apply(ys, order, weights) if _differentiable(ys, weights) else _combine(ys, order, weights)


# ---------------------------------------------------------------- products

def _forward(x, xld, weight, bias, gate, order, keep):
    """H and, with `keep`, the pre-activations of a gate."""
    L = experts_lib()
    (P, K), (n, N, _) = x.shape, weight.shape
    out = N // 2 if gate >= 0 else N
    h = x.new_empty((P, out))
    z = x.new_empty((P, 2 * (-(-out // 8) * 8)), dtype=torch.float32) if keep and gate >= 0 else None
    ok(L.sgemm_emu_expert_linear(DTYPES[x.dtype], P, N, K, n, addr(x), xld, addr(weight), addr(bias), gate,
                                 addr(order.offsets), addr(h), max(out, 1), addr(z), stream_of(x.get_device())),
       "sgemm_emu_expert_linear")
    return h, z


class _ExpertFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, gate, order):
        x, xld = rows_of(x)
        weight = weight.contiguous()
        bias = None if bias is None else bias.contiguous()
        h, z = _forward(x, xld, weight, bias, gate, order, True)
        # rows are read by the weight's gradient alone, the weight by the rows' alone
        need_x, need_w, _ = ctx.needs_input_grad[:3]
        ctx.save_for_backward(x if need_w else None, weight if need_x else None, z)
        ctx.gate, ctx.order, ctx.has_bias, ctx.dims = gate, order, bias is not None, (*weight.shape, x.shape[0])
        return h

    @staticmethod
    @once
    def backward(ctx, dh):
        x, weight, z = ctx.saved_tensors
        gate, order = ctx.gate, ctx.order
        need_x, need_w, need_b = ctx.needs_input_grad[:3]
        need_b = need_b and ctx.has_bias
        L = experts_lib()
        dt = DTYPES[dh.dtype]
        n, N, K, P = ctx.dims
        (x, xld), (dh, dhld) = (None, max(K, 1)) if x is None else rows_of(x), rows_of(dh)
        dx = dh.new_empty((P, K)) if need_x else None
        dw = dh.new_empty((n, N, K)) if need_w else None
        db = dh.new_empty((n, N)) if need_b else None
        nws = ok(L.sgemm_emu_expert_linear_backward_workspace(dt, P, N, K, n, gate, need_b),
                 "sgemm_emu_expert_linear_backward_workspace")
        ws = scratch(nws, dh)
        ok(L.sgemm_emu_expert_linear_backward(dt, P, N, K, n, addr(x), xld, addr(weight), addr(z), gate,
                                              addr(order.offsets), addr(dh), dhld, addr(dx), max(K, 1), addr(dw),
                                              addr(db), addr(ws), nws, stream_of(dh.get_device())),
           "sgemm_emu_expert_linear_backward")
        return dx, dw, db, None, None


def gate_code(gate, rows):
    """The library's number of a gate (None: none) of a weight of `rows` rows."""
    if gate is None:
        return SGEMM_EMU_GATE_NONE
    act = GATES.get(gate)
    if act is None:
        raise ValueError(f"unknown gate {gate!r} (one of {', '.join(GATES)}, or None)")
    if rows % 2 != 0:
        raise ValueError(f"weight: expected an even number of rows (gate, then up), got {rows}")
    return act


def expert_linear(x, weight, order, bias=None, gate=None):
    """On the rows of expert e (order.offsets): x weight[e]^T + bias[e], or with a gate ("silu", "gelu",
    "gelu_tanh", "sigmoid", "relu") act(x Wg^T + bg) * (x Wu^T + bu), weight[e] = [Wg; Wu]; zeros on rows of
    no expert.  x [T k, K] sorted (gather_tokens), weight [n, N, K], bias [n, N] or None, all float32 or all
    bfloat16 on the current HIP device.  Differentiable in x, weight and bias, in reverse mode; of a bfloat16 gate,
    the gradients of x and weight are products of its pre-activations' gradient rounded to bfloat16."""
    if not _fits(x, order, getattr(order, "rows", None)):
        check_order(order)
        check_tensor(x, "x", value_type(x, "x"), (order.rows, None))
    dt = x.dtype
    check_tensor(weight, "weight", dt, (order.experts, None, x.shape[1]))
    if bias is not None:
        check_tensor(bias, "bias", dt, weight.shape[:2])
    act = gate_code(gate, weight.shape[1])
    if _differentiable(x, weight, bias):
        return _ExpertFn.apply(x, weight, bias, act, order)
    x, xld = rows_of(x)
    return _forward(x, xld, weight.contiguous(), None if bias is None else bias.contiguous(), act, order, False)[0]


class ExpertFeedForward(torch.nn.Module):
    """A gated feed-forward layer of experts: forward(x [T, K], ids [T, k], weights [T, k] or None) is the sum
    over a token's experts of weights[t, j] down_e(act(gate_e x) * up_e x).  `up` [n, 2 hidden, features] (gate
    rows, then up rows) and `down` [n, features, hidden], with `up_bias` and `down_bias`, are trainable; which
    experts a token takes and their weights (of a router) are the caller's."""

    def __init__(self, features, hidden, experts, bias=False, gate="silu", device=None, dtype=None):
        super().__init__()
        if gate not in GATES:
            raise ValueError(f"unknown gate {gate!r} (one of {', '.join(GATES)})")
        self.features, self.hidden, self.experts, self.gate = features, hidden, experts, gate
        kw = {"device": device, "dtype": dtype}
        self.up = torch.nn.Parameter(torch.empty((experts, 2 * hidden, features), **kw))
        self.down = torch.nn.Parameter(torch.empty((experts, features, hidden), **kw))
        self.up_bias = torch.nn.Parameter(torch.zeros((experts, 2 * hidden), **kw)) if bias else None
        self.down_bias = torch.nn.Parameter(torch.zeros((experts, features), **kw)) if bias else None
        for w in (self.up, self.down):
            bound = w.shape[2] ** -0.5 if w.shape[2] else 0.0
            torch.nn.init.uniform_(w, -bound, bound)

    def forward(self, x, ids, weights=None):
        order = sort_tokens(ids, self.experts)
        h = expert_linear(gather_tokens(x, order), self.up, order, self.up_bias, self.gate)
        return combine_tokens(expert_linear(h, self.down, order, self.down_bias), order, weights)

    def extra_repr(self):
        return (f"features={self.features}, hidden={self.hidden}, experts={self.experts}, "
                f"bias={self.up_bias is not None}, gate={self.gate}")
