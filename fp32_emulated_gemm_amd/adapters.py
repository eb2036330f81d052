"""A fixed linear layer with low-rank adapters, many of them in one call, for
float32 tensors on the emulated GEMM and for bfloat16 tensors:

    Y[t] = W X[t] + bias + scale[i] up_i (down_i X[t]),   i = ids[t]

Rows of any order and mixture of adapters, or none (an id outside [0, n)): the
requests of a batch, each with its own fine-tuned adapter, share the product with
W.  Differentiable in x and the adapters (fine-tuning beside a fixed weight);
gradients are deterministic.
"""
import torch

from . import ops
from .ops import (DTYPES, FixedWeight, WeightPlan, addr, check_tensor, few_bytes, forward_mode, ok, ops_lib, rows_of,
                  scratch, stream_of)


def plan_weight(weight, backward=False):
    """The layout of a fixed weight for adapter_linear's `plan`; backward: W^T's too, for gradients
    (see ops.WeightPlan)."""
    return WeightPlan(weight, backward=backward)


def _forward(x, xld, weight, wld, a, b, ids, scale, bias, plan, keep):
    """Y and, with `keep`, the low-rank activations S."""
    L = ops_lib()
    dt = DTYPES[x.dtype]
    (M, K), N, (n, r, _) = x.shape, weight.shape[0], a.shape
    y = x.new_empty((M, N))
    s = x.new_empty((M, -(-r // 16) * 16), dtype=torch.float32) if keep and n > 0 and r > 0 else None
    fwd = None if plan is None else addr(plan.forward)
    xp, wp, bp, sp = addr(x), addr(weight), addr(b), addr(s)

    def query():
        return L.sgemm_emu_adapter_linear_workspace(dt, M, N, K, xp, xld, wp, wld, fwd, n, r, bp, sp)

    if M <= ops.FEW_ROWS and s is None:
        nws = few_bytes((dt, M, N, K, n > 0, r, x.device), query)
    else:
        nws = ok(query(), "sgemm_emu_adapter_linear_workspace")
    ws = scratch(nws, x)
    ok(L.sgemm_emu_adapter_linear(dt, M, N, K, xp, xld, wp, wld, fwd, addr(bias), n, r, addr(a), bp, addr(scale),
                                  addr(ids), addr(y), max(N, 1), sp, addr(ws), nws, stream_of(x.get_device())),
       "sgemm_emu_adapter_linear")
    return y, s


class _AdapterFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, a, b, ids, scale, bias, plan):
        x, xld = rows_of(x)
        weight, wld = rows_of(weight)
        a, b, ids = a.contiguous(), b.contiguous(), ids.contiguous()
        y, s = _forward(x, xld, weight, wld, a, b, ids, scale, bias, plan, True)
        ctx.save_for_backward(x, weight, a, b, ids, scale, s)
        ctx.plan = plan
        return y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        need_x, need_w, need_a, need_b, _, need_scale, need_bias = ctx.needs_input_grad[:7]
        if need_w or need_bias or need_scale:
            raise RuntimeError("fp32_emulated_gemm_amd.adapters provides the gradients of x and the adapters only; "
                               "set requires_grad=False on the weight, the bias and the scale")
        x, weight, a, b, ids, scale, s = ctx.saved_tensors
        L = ops_lib()
        dt = DTYPES[x.dtype]
        (M, K), N, (n, r, _) = x.shape, weight.shape[0], a.shape
        (x, xld), (dy, dyld) = rows_of(x), rows_of(dy)
        back = None
        if need_x:
            plan = ctx.plan
            if plan is None or plan.backward is None:
                plan = WeightPlan(weight, forward=False, backward=True)
            back = plan.backward
        dx = x.new_empty((M, K)) if need_x else None
        da = torch.empty_like(a) if need_a else None
        db = torch.empty_like(b) if need_b else None
        nws = ok(L.sgemm_emu_adapter_linear_backward_workspace(dt, M, N, K, n, r),
                 "sgemm_emu_adapter_linear_backward_workspace")
        ws = scratch(nws, x)
        ok(L.sgemm_emu_adapter_linear_backward(dt, M, N, K, addr(x), xld, addr(back), n, r, addr(a), addr(b),
                                               addr(scale), addr(ids), addr(s), addr(dy), dyld, addr(dx), max(K, 1),
                                               addr(da), addr(db), addr(ws), nws, stream_of(x.get_device())),
           "sgemm_emu_adapter_linear_backward")
        return dx, None, da, db, None, None, None, None


def _check(x, weight, a, b, ids, scale, bias):
    """Raises for the first argument that does not fit."""
    if not isinstance(x, torch.Tensor):
        raise TypeError(f"x: expected a torch tensor, got {type(x).__name__}")
    dt = x.dtype
    if dt not in DTYPES:
        raise TypeError(f"x: expected dtype float32 or bfloat16, got {dt}")
    if x.dim() < 1:
        raise ValueError("x: expected at least one dimension")
    check_tensor(x, "x", dt, x.shape)
    check_tensor(weight, "weight", dt, (None, x.shape[-1]))
    check_tensor(a, "a", dt, (None, None, x.shape[-1]))
    check_tensor(b, "b", dt, (a.shape[0], weight.shape[0], a.shape[1]))
    check_tensor(ids, "ids", torch.int32, x.shape[:-1])
    if bias is not None:
        check_tensor(bias, "bias", dt, (weight.shape[0],))
    if scale is not None:
        check_tensor(scale, "scale", torch.float32, (a.shape[0],))


def _fits(x, weight, a, b, ids, scale, bias):
    """Whether every argument fits: _check's conditions in one expression, for the calls where the
    host's time counts (1 us instead of 8)."""
    dt, shape, d = x.dtype, x.shape, torch.cuda.current_device()
    N, K = weight.shape
    n, r, Ka = a.shape
    return (dt in DTYPES and weight.dtype is dt and a.dtype is dt and b.dtype is dt and ids.dtype is torch.int32
            and shape[-1] == K == Ka and b.shape == (n, N, r) and ids.shape == shape[:-1]
            and x.get_device() == d == weight.get_device() == a.get_device() == b.get_device() == ids.get_device()
            and (bias is None or (bias.dtype is dt and bias.shape == (N,) and bias.get_device() == d))
            and (scale is None or (scale.dtype is torch.float32 and scale.shape == (n,) and scale.get_device() == d)))


def adapter_linear(x, weight, a, b, ids, scale=None, bias=None, plan=None):
    """x W^T + bias + scale[i] (x a[i]^T) b[i]^T with i = ids[row], for x[..., K], weight[N, K],
    a[n, r, K], b[n, N, r], bias[N] or None, all float32 or all bfloat16 on the current HIP device;
    ids: int32 of x's leading shape (outside [0, n): no adapter); scale: None (1), a number, or float32
    [n].  `plan` (plan_weight(weight)) spares laying the weight out.  Differentiable in x, a and b, in reverse
    mode."""
    if scale is not None and not isinstance(scale, torch.Tensor) and isinstance(a, torch.Tensor):
        scale = torch.full(a.shape[:1], float(scale), dtype=torch.float32, device=a.device)
    try:
        fits = _fits(x, weight, a, b, ids, scale, bias)
    except (AttributeError, IndexError, TypeError, ValueError, RuntimeError):   # RuntimeError: no device
        fits = False
    if not fits:
        _check(x, weight, a, b, ids, scale, bias)
    dims, K, N = x.dim(), x.shape[-1], weight.shape[0]
    if plan is not None:
        plan.check(weight, gated=False)
    x2d = x if dims == 2 else x.reshape(x.shape[:-1].numel(), K)
    if ids.dim() != 1:
        ids = ids.reshape(-1)
    ops_lib()
    bias = None if bias is None else bias.contiguous()
    scale = None if scale is None else scale.contiguous()
    if forward_mode() or (torch.is_grad_enabled()
                          and (x.requires_grad or a.requires_grad or b.requires_grad or weight.requires_grad
                               or (scale is not None and scale.requires_grad)
                               or (bias is not None and bias.requires_grad))):
        y = _AdapterFn.apply(x2d, weight, a, b, ids, scale, bias, plan)
    else:
        (xr, xld), (wr, wld) = rows_of(x2d), rows_of(weight)
        y, _ = _forward(xr, xld, wr, wld, a.contiguous(), b.contiguous(), ids.contiguous(), scale, bias, plan, False)
    return y if dims == 2 else y.reshape(*x.shape[:-1], N)


class AdapterLinear(torch.nn.Module):
    """A fixed linear layer with `adapters` trainable low-rank adapters of rank `rank`:
    forward(x, ids).  `up` starts at zero, so a new adapter changes nothing.  Every call reads the
    weight as it is; `plan` (plan_weight(m.weight, backward=True)) spares laying it out where the
    caller knows that it does not change."""

    def __init__(self, in_features, out_features, adapters, rank, alpha=None, bias=True, device=None, dtype=None):
        super().__init__()
        self.in_features, self.out_features = in_features, out_features
        self.adapters, self.rank = adapters, rank
        kw = {"device": device, "dtype": dtype}
        self.weight = torch.nn.Parameter(torch.empty((out_features, in_features), **kw), requires_grad=False)
        self.bias = torch.nn.Parameter(torch.zeros(out_features, **kw), requires_grad=False) if bias else None
        self.down = torch.nn.Parameter(torch.empty((adapters, rank, in_features), **kw))
        self.up = torch.nn.Parameter(torch.zeros((adapters, out_features, rank), **kw))
        self.register_buffer("scale", torch.full((adapters,), 1.0 if alpha is None else alpha / max(rank, 1),
                                                 dtype=torch.float32, device=device))
        bound = in_features ** -0.5 if in_features else 0.0
        torch.nn.init.uniform_(self.weight, -bound, bound)
        torch.nn.init.uniform_(self.down, -bound, bound)
        self._fixed = None

    @classmethod
    def from_linear(cls, layer, adapters, rank, alpha=None):
        """The weights of a torch.nn.Linear (or this package's Linear), fixed, with fresh adapters."""
        m = cls(layer.in_features, layer.out_features, adapters, rank, alpha, layer.bias is not None,
                layer.weight.device, layer.weight.dtype)
        with torch.no_grad():
            m.weight.copy_(layer.weight)
            if layer.bias is not None:
                m.bias.copy_(layer.bias)
        return m.fix_weights()

    def _apply(self, fn, recurse=True):
        """Moves and casts as Module does, but the scale, which the kernels take in 32 bits, keeps its
        type and its value."""
        scale = self.scale
        super()._apply(fn, recurse)
        if self.scale.dtype != scale.dtype:
            self.scale = scale.to(self.scale.device)
        return self

    def fix_weights(self):
        """Take the weight as it is for the fixed one: calls raise once it has changed, until this is
        called again."""
        self._fixed = FixedWeight(self.weight)
        return self

    def forward(self, x, ids, plan=None):
        if self._fixed is not None:
            self._fixed.check(self.weight)
        return adapter_linear(x, self.weight, self.down, self.up, ids, self.scale, self.bias, plan)

    def extra_repr(self):
        return (f"in_features={self.in_features}, out_features={self.out_features}, adapters={self.adapters}, "
                f"rank={self.rank}, bias={self.bias is not None}")
