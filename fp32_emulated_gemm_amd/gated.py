"""The gated feed-forward projection of a transformer block (forward, input and
parameter gradients), for float32 tensors on the emulated GEMM and for bfloat16
tensors:

    H = act(Z[:, :F]) * Z[:, F:],   Z = X W^T + bias,

W [2F, K]: the gate's F rows, then the up projection's F rows.  Both projections,
the activation and the product are one call (sgemm_emu_gated_linear); the
backward pass (sgemm_emu_gated_linear_backward) is deterministic.
"""
import torch

from . import ops
from .linear import Linear
from .ops import (DTYPES, GATES, FixedWeight, WeightPlan, addr, check_tensor, few_bytes, forward_mode, ok, ops_lib,
                  rows_of, scratch, stream_of)


def plan_weight(weight):
    """The layout of a fixed weight for gated_linear's `plan` (see ops.WeightPlan)."""
    return WeightPlan(weight, gated=True)


def _forward(x, xld, weight, wld, bias, gate, plan, keep):
    """H and, with `keep`, the pre-activations Z."""
    L = ops_lib()
    dt = DTYPES[x.dtype]
    (M, K), F = x.shape, weight.shape[0] // 2
    h = x.new_empty((M, F))
    z = x.new_empty((M, 2 * (-(-F // 8) * 8)), dtype=torch.float32) if keep else None
    fwd = None if plan is None else addr(plan.forward)
    xp, wp, zp = addr(x), addr(weight), addr(z)

    def query():
        return L.sgemm_emu_gated_linear_workspace(dt, M, F, K, xp, xld, wp, wld, fwd, zp)

    if M <= ops.FEW_ROWS and K and not keep:
        nws = few_bytes((dt, M, F, K, x.device), query)
    else:
        nws = ok(query(), "sgemm_emu_gated_linear_workspace")
    ws = scratch(nws, x)
    ok(L.sgemm_emu_gated_linear(dt, M, F, K, xp, xld, wp, wld, fwd, addr(bias), gate, addr(h), max(F, 1), zp,
                                addr(ws), nws, stream_of(x.get_device())), "sgemm_emu_gated_linear")
    return h, z


class _GatedFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, gate, plan):
        x, xld = rows_of(x)
        weight, wld = rows_of(weight)
        bias = None if bias is None else bias.contiguous()
        h, z = _forward(x, xld, weight, wld, bias, gate, plan, True)
        ctx.save_for_backward(x, weight, z)
        ctx.gate, ctx.has_bias = gate, bias is not None
        return h

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dh):
        x, weight, z = ctx.saved_tensors
        need_x, need_w, need_b = ctx.needs_input_grad[:3]
        L = ops_lib()
        dt = DTYPES[x.dtype]
        (M, K), F = x.shape, weight.shape[0] // 2
        (x, xld), (weight, wld), (dh, dhld) = rows_of(x), rows_of(weight), rows_of(dh)
        dx = x.new_empty((M, K)) if need_x else None
        dw = x.new_empty((2 * F, K)) if need_w else None
        db = x.new_empty((2 * F,)) if need_b and ctx.has_bias else None
        nws = ok(L.sgemm_emu_gated_linear_backward_workspace(dt, M, F, K), "sgemm_emu_gated_linear_backward_workspace")
        ws = scratch(nws, x)
        ok(L.sgemm_emu_gated_linear_backward(dt, M, F, K, addr(x), xld, addr(weight), wld, addr(z),
                                             ctx.gate, addr(dh), dhld, addr(dx), max(K, 1), addr(dw), max(K, 1),
                                             addr(db), addr(ws), nws, stream_of(x.get_device())),
           "sgemm_emu_gated_linear_backward")
        return dx, dw, db, None, None


def _check(x, weight, bias):
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
    if weight.shape[0] % 2 != 0:
        raise ValueError(f"weight: expected an even number of rows (gate, then up), got {weight.shape[0]}")
    if bias is not None:
        check_tensor(bias, "bias", dt, (weight.shape[0],))


def _fits(x, weight, bias):
    """Whether every argument fits: _check's conditions in one expression, for the calls where the
    host's time counts."""
    dt, d = x.dtype, torch.cuda.current_device()
    rows, K = weight.shape
    return (dt in DTYPES and weight.dtype is dt and x.shape[-1] == K and rows % 2 == 0
            and x.get_device() == d == weight.get_device()
            and (bias is None or (bias.dtype is dt and bias.shape == (rows,) and bias.get_device() == d)))


def gated_linear(x, weight, bias=None, gate="silu", plan=None):
    """act(x Wg^T + bg) * (x Wu^T + bu) for x[..., K], weight[2F, K] = [Wg; Wu], bias[2F] or None,
    all float32 or all bfloat16 on the current HIP device.  gate: "silu", "gelu" (exact), "gelu_tanh",
    "sigmoid" or "relu".  `plan` (plan_weight(weight)) spares laying out a weight that does not change.
    Differentiable in x, weight and bias, in reverse mode."""
    act = GATES.get(gate)
    if act is None:
        raise ValueError(f"unknown gate {gate!r} (one of {', '.join(GATES)})")
    try:
        fits = _fits(x, weight, bias)
    except (AttributeError, IndexError, TypeError, ValueError, RuntimeError):   # RuntimeError: no device
        fits = False
    if not fits:
        _check(x, weight, bias)
    dims, K, rows = x.dim(), x.shape[-1], weight.shape[0]
    x2d = x if dims == 2 else x.reshape(x.shape[:-1].numel(), K)
    if plan is not None:
        plan.check(weight, gated=True)
    ops_lib()
    if forward_mode() or (torch.is_grad_enabled() and (x.requires_grad or weight.requires_grad
                                                       or (bias is not None and bias.requires_grad))):
        h = _GatedFn.apply(x2d, weight, bias, act, plan)
    else:
        (xr, xld), (wr, wld) = rows_of(x2d), rows_of(weight)
        h, _ = _forward(xr, xld, wr, wld, None if bias is None else bias.contiguous(), act, plan, False)
    return h if dims == 2 else h.reshape(*x.shape[:-1], rows // 2)


class GatedLinear(torch.nn.Module):
    """gated_linear as a module: `weight` [2 out_features, in_features] (gate rows, then up rows) and
    `bias` [2 out_features], trainable.  fix_weights() freezes them.  Every call reads the weight as it
    is; `plan` (plan_weight(m.weight)) spares laying it out where the caller knows that it does not
    change."""

    def __init__(self, in_features, out_features, bias=True, gate="silu", device=None, dtype=None):
        super().__init__()
        if gate not in GATES:
            raise ValueError(f"unknown gate {gate!r} (one of {', '.join(GATES)})")
        self.in_features, self.out_features, self.gate = in_features, out_features, gate
        self.weight = torch.nn.Parameter(torch.empty((2 * out_features, in_features), device=device, dtype=dtype))
        self.bias = torch.nn.Parameter(torch.zeros(2 * out_features, device=device, dtype=dtype)) if bias else None
        self._fixed = None
        bound = in_features ** -0.5 if in_features else 0.0
        torch.nn.init.uniform_(self.weight, -bound, bound)

    @classmethod
    def from_linears(cls, gate_proj, up_proj, gate="silu"):
        """From two torch.nn.Linear layers of one shape: act(gate_proj(x)) * up_proj(x)."""
        if gate_proj.weight.shape != up_proj.weight.shape or (gate_proj.bias is None) != (up_proj.bias is None):
            raise ValueError("gate_proj and up_proj differ in shape or bias")
        m = cls(gate_proj.in_features, gate_proj.out_features, gate_proj.bias is not None, gate,
                gate_proj.weight.device, gate_proj.weight.dtype)
        with torch.no_grad():
            m.weight.copy_(torch.cat((gate_proj.weight, up_proj.weight)))
            if m.bias is not None:
                m.bias.copy_(torch.cat((gate_proj.bias, up_proj.bias)))
        return m

    def fix_weights(self):
        """Freeze the parameters: calls raise once the weight has changed, until this is called again."""
        for p in self.parameters():
            p.requires_grad_(False)
        self._fixed = FixedWeight(self.weight)
        return self

    def forward(self, x, plan=None):
        if self._fixed is not None:
            self._fixed.check(self.weight)
        return gated_linear(x, self.weight, self.bias, self.gate, plan)

    def extra_repr(self):
        return (f"in_features={self.in_features}, out_features={self.out_features}, "
                f"bias={self.bias is not None}, gate={self.gate}")


class GatedFeedForward(torch.nn.Module):
    """A float32 feed-forward block on the emulated GEMM: GatedLinear, then a fixed-weight Linear
    (down projection)."""

    def __init__(self, features, hidden, bias=True, gate="silu", device=None):
        super().__init__()
        self.up = GatedLinear(features, hidden, bias, gate, device, torch.float32)
        self.down = Linear(hidden, features, bias, device=device)

    @classmethod
    def from_linears(cls, gate_proj, up_proj, down_proj, gate="silu"):
        m = cls.__new__(cls)
        torch.nn.Module.__init__(m)
        m.up = GatedLinear.from_linears(gate_proj, up_proj, gate)
        m.down = Linear.from_linear(down_proj)
        return m

    def forward(self, x):
        return self.down(self.up(x))
