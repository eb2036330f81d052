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
from .ops import WeightPlan, addr, check_tensor, current_stream, ok, ops_lib, rows_of, scratch


def plan_weight(weight, backward=False):
    """The layout of a fixed weight for adapter_linear's `plan`; backward: W^T's too, for gradients
    (see ops.WeightPlan)."""
    return WeightPlan(weight, backward=backward)


def _forward(x, xld, weight, wld, a, b, ids, scale, bias, plan, keep):
    """Y and, with `keep`, the low-rank activations S."""
    L = ops_lib()
    dt = ops.DTYPES[x.dtype]
    (M, K), N, (n, r) = x.shape, weight.shape[0], a.shape[:2]
    y = torch.empty((M, N), dtype=x.dtype, device=x.device)
    low = n > 0 and r > 0
    s = torch.empty((M, -(-r // 16) * 16), dtype=torch.float32, device=x.device) if low and keep else None
    fwd = None if plan is None else addr(plan.forward)
    xp, wp, bp, sp = addr(x), addr(weight), addr(b), addr(s)
    ws, nws = scratch(ok(L.sgemm_emu_adapter_linear_workspace(dt, M, N, K, xp, xld, wp, wld, fwd, n, r, bp, sp),
                             "sgemm_emu_adapter_linear_workspace"), x.device)
    ok(L.sgemm_emu_adapter_linear(dt, M, N, K, xp, xld, wp, wld, fwd, addr(bias), n, r, addr(a), bp, addr(scale),
                                  addr(ids), addr(y), max(N, 1), sp, addr(ws), nws, current_stream()),
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
        dt = ops.DTYPES[x.dtype]
        (M, K), N, (n, r) = x.shape, weight.shape[0], a.shape[:2]
        (x, xld), (dy, dyld) = rows_of(x), rows_of(dy)
        back = None
        if need_x:
            plan = ctx.plan
            if plan is None or plan.backward is None:
                plan = WeightPlan(weight, forward=False, backward=True)
            back = plan.backward
        dx = torch.empty((M, K), dtype=x.dtype, device=x.device) if need_x else None
        da = torch.empty_like(a) if need_a else None
        db = torch.empty_like(b) if need_b else None
        ws, nws = scratch(ok(L.sgemm_emu_adapter_linear_backward_workspace(dt, M, N, K, n, r),
                             "sgemm_emu_adapter_linear_backward_workspace"), x.device)
        ok(L.sgemm_emu_adapter_linear_backward(dt, M, N, K, addr(x), xld, addr(back), n, r, addr(a), addr(b),
                                               addr(scale), addr(ids), addr(s), addr(dy), dyld, addr(dx), max(K, 1),
                                               addr(da), addr(db), addr(ws), nws, current_stream()),
           "sgemm_emu_adapter_linear_backward")
        return dx, None, da, db, None, None, None, None


def adapter_linear(x, weight, a, b, ids, scale=None, bias=None, plan=None):
    """x W^T + bias + scale[i] (x a[i]^T) b[i]^T with i = ids[row], for x[..., K], weight[N, K],
    a[n, r, K], b[n, N, r], bias[N] or None, all float32 or all bfloat16 on the current HIP device;
    ids: int32 of x's leading shape (outside [0, n): no adapter); scale: None (1), a number, or float32
    [n].  `plan` (plan_weight(weight)) spares laying the weight out.  Differentiable in x, a and b."""
    for name, t in (("x", x), ("weight", weight), ("a", a), ("b", b), ("ids", ids)):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name}: expected a torch tensor, got {type(t).__name__}")
    dt = x.dtype
    if dt not in ops.DTYPES:
        raise TypeError(f"x: expected dtype float32 or bfloat16, got {dt}")
    if x.dim() < 1:
        raise ValueError("x: expected at least one dimension")
    K = x.shape[-1]
    check_tensor(weight, "weight", dt, (None, K))
    N = weight.shape[0]
    check_tensor(a, "a", dt, (None, None, K))
    n, r = a.shape[:2]
    check_tensor(b, "b", dt, (n, N, r))
    check_tensor(ids, "ids", torch.int32, x.shape[:-1])
    if bias is not None:
        check_tensor(bias, "bias", dt, (N,))
    if scale is not None and not isinstance(scale, torch.Tensor):
        scale = torch.full((n,), float(scale), dtype=torch.float32, device=x.device)
    if scale is not None:
        check_tensor(scale, "scale", torch.float32, (n,))
        scale = scale.contiguous()
    if plan is not None:
        plan.check(weight)
    x2d = x if x.dim() == 2 else x.reshape(-1, K) if K else x.new_empty(x.shape[:-1].numel(), 0)
    check_tensor(x2d, "x", dt, (None, None))
    if ids.dim() != 1:
        ids = ids.reshape(-1)
    ops_lib()
    bias = None if bias is None else bias.contiguous()
    if torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in (x, weight, a, b, scale, bias)):
        y = _AdapterFn.apply(x2d, weight, a, b, ids, scale, bias, plan)
    else:
        (xr, xld), (wr, wld) = rows_of(x2d), rows_of(weight)
        y, _ = _forward(xr, xld, wr, wld, a.contiguous(), b.contiguous(), ids.contiguous(), scale, bias, plan, False)
    return y if x.dim() == 2 else y.reshape(*x.shape[:-1], N)


class AdapterLinear(torch.nn.Module):
    """A fixed linear layer with `adapters` trainable low-rank adapters of rank `rank`:
    forward(x, ids).  `up` starts at zero, so a new adapter changes nothing."""

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
        self._plan = None

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

    def fix_weights(self):
        """Lay the weight out (after it was loaded or changed)."""
        self._plan = (plan_weight(self.weight, backward=True), self.weight._version)
        return self

    def forward(self, x, ids):
        plan = None
        if self._plan is not None:
            plan, version = self._plan
            if version != self.weight._version or plan.device != self.weight.device:
                raise RuntimeError("the weight changed after fix_weights(); call it again")
        return adapter_linear(x, self.weight, self.down, self.up, ids, self.scale, self.bias, plan)

    def extra_repr(self):
        return (f"in_features={self.in_features}, out_features={self.out_features}, adapters={self.adapters}, "
                f"rank={self.rank}, bias={self.bias is not None}")
