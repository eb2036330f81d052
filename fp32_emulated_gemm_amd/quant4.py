"""Layers and experts served with weights of 4 bits: each value stands for
(q - zero) scale, scale and zero shared by a group of 32, 64 or 128 columns of a row.

    w4 = quantize(weight)                       # [N, K], or [n, N, K] of experts
    y = quant4_linear(x, w4, bias)              # x [..., K]
    h = quant4_linear(xs, w4, gate="silu", order=order)     # experts, on sorted rows

A few rows (single tokens: up to 64, float32 with groups of 64 or 128 up to 128, or 16 an
expert) read the packed weights in one pass and sum (q - zero) x in 32 bits.  Longer calls
unpack them first, rounded to the rows' type: in bfloat16 the weight then has 8 bits, and the
outputs' relative error is 0.0024 where it is 0.0017 with few rows.  Forward only: weights of
4 bits are served, not trained.  The calls are those of include/sgemm_emu_experts.h.
"""
import torch

from . import ops
from .adapters import AdapterLinear
from .experts import (ExpertFeedForward, check_order, combine_tokens, experts_lib, gate_code, gather_tokens,
                      sort_tokens, value_type)
from .ops import DTYPES, addr, check_tensor, forward_mode, ok, rows_of, scratch, stream_of

GROUPS = (32, 64, 128)


class Quant4Weight:
    """A weight [N, K] or a bank of experts' [n, N, K] held in 4 bits, laid out by quantize or pack."""

    __slots__ = ("packed", "shape", "group", "zeros", "bank")

    def __init__(self, packed, shape, group, zeros):
        self.packed, self.shape, self.group, self.zeros = packed, tuple(shape), group, zeros
        # (experts, rows, columns), one expert for a layer's weight
        self.bank = self.shape if len(self.shape) == 3 else (1, *self.shape)

    def dequantize(self, dtype=torch.float32):
        """The weights that it stands for, rounded to `dtype` (float32 or bfloat16)."""
        if dtype not in DTYPES:
            raise TypeError(f"dtype: expected float32 or bfloat16, got {dtype}")
        check_tensor(self.packed, "packed", torch.uint8, (None,))
        w = torch.empty(self.shape, dtype=dtype, device=self.packed.device)
        ok(experts_lib().sgemm_emu_quant4_unpack(DTYPES[dtype], *self.bank, self.group, self.zeros,
                                                 addr(self.packed), addr(w), stream_of(w.get_device())),
           "sgemm_emu_quant4_unpack")
        return w


def _check_group(group):
    if group not in GROUPS:
        raise ValueError(f"group: expected one of {GROUPS}, got {group}")


def _bank(shape):
    if len(shape) not in (2, 3):
        raise ValueError(f"expected a weight of two or three dimensions, got {len(shape)}")
    return tuple(shape) if len(shape) == 3 else (1, *shape)


def pack(q, scale, zero=None, group=128):
    """The weights (q - zero) scale laid out for quant4_linear: q uint8 0..15 [N, K] or [n, N, K]; scale float32
    and zero uint8 0..15 (None: 8) [..., N, ceil(K / group)]."""
    _check_group(group)
    if not isinstance(q, torch.Tensor):
        raise TypeError(f"q: expected a torch tensor, got {type(q).__name__}")
    bank = _bank(q.shape)
    check_tensor(q, "q", torch.uint8, q.shape)
    groups = (*q.shape[:-1], -(-q.shape[-1] // group))
    check_tensor(scale, "scale", torch.float32, groups)
    if zero is not None:
        check_tensor(zero, "zero", torch.uint8, groups)
    L = experts_lib()
    q, scale = q.contiguous(), scale.detach().contiguous()
    zero = None if zero is None else zero.contiguous()
    nbytes = ok(L.sgemm_emu_quant4_bytes(*bank, group, zero is not None), "sgemm_emu_quant4_bytes")
    packed = q.new_empty(max(nbytes, 16))
    ok(L.sgemm_emu_quant4_pack(*bank, group, addr(q), addr(scale), addr(zero), packed.data_ptr(),
                               stream_of(q.get_device())), "sgemm_emu_quant4_pack")
    return Quant4Weight(packed, q.shape, group, zero is not None)


def quantize_values(weight, group=128, symmetric=False):
    """(q, scale, zero) nearest to weight [N, K] or [n, N, K] (float32 or bfloat16); zero is None if symmetric."""
    _check_group(group)
    dt = value_type(weight, "weight")
    bank = _bank(weight.shape)
    check_tensor(weight, "weight", dt, weight.shape)
    w = weight.detach().contiguous()
    q = torch.empty(w.shape, dtype=torch.uint8, device=w.device)
    groups = (*w.shape[:-1], -(-w.shape[-1] // group))
    scale = torch.empty(groups, dtype=torch.float32, device=w.device)
    zero = None if symmetric else torch.empty(groups, dtype=torch.uint8, device=w.device)
    ok(experts_lib().sgemm_emu_quant4_quantize(DTYPES[dt], *bank, group, addr(w), addr(q), addr(scale), addr(zero),
                                               stream_of(w.get_device())), "sgemm_emu_quant4_quantize")
    return q, scale, zero


def quantize(weight, group=128, symmetric=False):
    """weight [N, K] or [n, N, K] (float32 or bfloat16) in 4 bits, each group rounded to nearest."""
    q, scale, zero = quantize_values(weight, group, symmetric)
    return pack(q, scale, zero, group)


def quant4_linear(x, weight, bias=None, gate=None, order=None):
    """x W^T + bias, or with a gate act(x Wg^T + bg) * (x Wu^T + bu), W = [Wg; Wu] the Quant4Weight `weight`.
    Without `order`: x [..., K], weight [N, K], bias [N].  With it (sort_tokens): x [T k, K] sorted, weight
    [n, N, K], bias [n, N], as in experts.expert_linear.  x and bias float32 or bfloat16; with more rows than
    read the packed weight, W is rounded to that type.  Forward only."""
    if not isinstance(weight, Quant4Weight):
        raise TypeError(f"weight: expected a Quant4Weight (of quantize or pack), got {type(weight).__name__}")
    dt = value_type(x, "x")
    n, N, K = weight.bank
    shape, d = x.shape, x.get_device()
    if order is None:
        if len(weight.shape) != 2:
            raise ValueError("weight: a bank of experts needs the rows' order")
        if len(shape) < 1:
            raise ValueError("x: expected at least one dimension")
        P = shape[0] if len(shape) == 2 else shape[:-1].numel()
    else:
        check_order(order)
        if len(weight.shape) != 3:
            raise ValueError("weight: one layer's weight takes no order")
        if n != order.experts:
            raise ValueError(f"weight: expected a bank of {order.experts} experts, got {n}")
        P = order.rows
    if not (x.is_cuda and shape[-1:] == (K,) and d == torch.cuda.current_device() and (order is None or tuple(shape) == (P, K))):
        check_tensor(x, "x", dt, (*shape[:-1], K) if order is None else (P, K))
    if bias is not None:
        check_tensor(bias, "bias", dt, (N,) if order is None else (n, N))
    if weight.packed.get_device() != d:
        raise ValueError(f"weight: expected one on {x.device}, got {weight.packed.device}")
    act = gate_code(gate, N)
    if torch.is_grad_enabled() and (x.requires_grad or (bias is not None and bias.requires_grad)):
        raise RuntimeError("quant4_linear is forward only: detach x and bias, or call it under torch.no_grad()")
    if forward_mode():
        for t in (x, bias):
            if t is not None and torch.autograd.forward_ad.unpack_dual(t).tangent is not None:
                raise NotImplementedError("quant4_linear has no forward-mode derivative")
    L = experts_lib()
    x2d, xld = rows_of(x if len(shape) == 2 else x.reshape(P, K))
    bias = None if bias is None else bias.contiguous()
    out = N // 2 if gate is not None else N
    h = x.new_empty((P, out))
    code = DTYPES[dt]
    nws = 0
    if P > ops.FEW_ROWS:                 # fewer read the packed weight
        nws = ok(L.sgemm_emu_quant4_linear_workspace(code, P, N, K, n, weight.group, weight.zeros),
                 "sgemm_emu_quant4_linear_workspace")
    ws = scratch(nws, x)
    ok(L.sgemm_emu_quant4_linear(code, P, N, K, n, weight.group, weight.zeros, addr(x2d), xld, addr(weight.packed),
                                 addr(bias), act, None if order is None else addr(order.offsets), addr(h),
                                 max(out, 1), addr(ws), nws, stream_of(d)), "sgemm_emu_quant4_linear")
    return h if len(shape) == 2 else h.reshape(*shape[:-1], out)


class _Held(torch.nn.Module):
    """A Quant4Weight and a bias as a module's buffers, which move and are saved with it."""

    def _hold(self, name, weight, bias):
        self.register_buffer(name, weight.packed)
        self.register_buffer(name + "_bias", None if bias is None else bias.detach().clone())
        setattr(self, "_" + name, (weight.shape, weight.group, weight.zeros))

    def _held(self, name):
        return Quant4Weight(getattr(self, name), *getattr(self, "_" + name))


class Quant4Linear(_Held):
    """A layer served in 4 bits, with or without a gate: forward(x)."""

    def __init__(self, weight, bias=None, gate=None):
        super().__init__()
        gate_code(gate, weight.shape[0])
        self.gate = gate
        self._hold("layer", weight, bias)

    @classmethod
    def from_linear(cls, layer, group=128, symmetric=False):
        """From a torch.nn.Linear, or this package's Linear or GatedLinear (its gate with it).  Layers that compute
        more, by a fused activation or adapters, are refused."""
        if getattr(layer, "activation", None) is not None:
            raise ValueError(f"layer: its activation {layer.activation!r} would be lost; apply it to the served layer's output")
        if isinstance(layer, AdapterLinear):
            raise ValueError("layer: its adapters would be lost; quantize its weight alone")
        return cls(quantize(layer.weight, group, symmetric), layer.bias, getattr(layer, "gate", None))

    @property
    def weight(self):
        return self._held("layer")

    def forward(self, x):
        return quant4_linear(x, self.weight, self.layer_bias, self.gate)

    def extra_repr(self):
        (N, K), group, _ = self._layer
        return f"in_features={K}, rows={N}, group={group}, bias={self.layer_bias is not None}, gate={self.gate}"


class Quant4ExpertFeedForward(_Held):
    """experts.ExpertFeedForward served in 4 bits: forward(x, ids, weights)."""

    def __init__(self, up, down, up_bias=None, down_bias=None, gate="silu"):
        super().__init__()
        gate_code(gate, up.shape[1])
        self.gate = gate
        self._hold("up", up, up_bias)
        self._hold("down", down, down_bias)

    @classmethod
    def from_experts(cls, layer: ExpertFeedForward, group=128, symmetric=False):
        return cls(quantize(layer.up, group, symmetric), quantize(layer.down, group, symmetric), layer.up_bias,
                   layer.down_bias, layer.gate)

    def forward(self, x, ids, weights=None):
        up, down = self._held("up"), self._held("down")
        order = sort_tokens(ids, up.shape[0])
        h = quant4_linear(gather_tokens(x, order), up, self.up_bias, self.gate, order)
        return combine_tokens(quant4_linear(h, down, self.down_bias, None, order), order, weights)

    def extra_repr(self):
        (n, _, K), group, _ = self._up
        return f"features={K}, experts={n}, group={group}, bias={self.up_bias is not None}, gate={self.gate}"
