"""Python binding of the operators in ``include/sgemm_emu_ops.h``: the gated
feed-forward projection and the linear layer with low-rank adapters.

Thin ctypes marshalling with the C names and argument order; every step runs in
the library's HIP kernels.  The tensor functions that check their arguments,
allocate outputs and differentiate are in ``gated`` and ``adapters``.
"""
import ctypes

import torch
from torch.autograd import forward_ad

from . import SgemmEmuError, lib

SGEMM_EMU_F32 = 0
SGEMM_EMU_BF16 = 1
SGEMM_EMU_GATE_SILU = 0
SGEMM_EMU_GATE_GELU = 1        # exact (erf) form
SGEMM_EMU_GATE_GELU_TANH = 2
SGEMM_EMU_GATE_SIGMOID = 3
SGEMM_EMU_GATE_RELU = 4
SGEMM_EMU_PLAN_ROWS = 0
SGEMM_EMU_PLAN_TRANSPOSED = 1
SGEMM_EMU_PLAN_GATED = 2

DTYPES = {torch.float32: SGEMM_EMU_F32, torch.bfloat16: SGEMM_EMU_BF16}
GATES = {"silu": SGEMM_EMU_GATE_SILU, "gelu": SGEMM_EMU_GATE_GELU, "gelu_tanh": SGEMM_EMU_GATE_GELU_TANH,
         "sigmoid": SGEMM_EMU_GATE_SIGMOID, "relu": SGEMM_EMU_GATE_RELU}

OPS_EXPORTS = ("sgemm_emu_plan_bytes", "sgemm_emu_plan_weight", "sgemm_emu_gated_linear_workspace",
               "sgemm_emu_gated_linear", "sgemm_emu_gated_linear_backward_workspace",
               "sgemm_emu_gated_linear_backward", "sgemm_emu_adapter_linear_workspace", "sgemm_emu_adapter_linear",
               "sgemm_emu_adapter_linear_backward_workspace", "sgemm_emu_adapter_linear_backward",
               "sgemm_emu_few_rows")

MAX_LD = 8388544   # leading dimensions that the library takes

_OPS = None
FEW_ROWS = None   # sgemm_emu_few_rows(), set when the library is first used


def ops_lib():
    """The library with the operators' signatures set (once)."""
    global _OPS, FEW_ROWS
    if _OPS is None:
        L = lib()
        i64, vp, ci = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int
        dims3 = [ci, i64, i64, i64]
        L.sgemm_emu_plan_bytes.argtypes = [ci, i64, i64, ci]
        L.sgemm_emu_plan_weight.argtypes = [ci, i64, i64, vp, i64, ci, vp, vp]
        L.sgemm_emu_gated_linear_workspace.argtypes = dims3 + [vp, i64, vp, i64, vp, vp]
        L.sgemm_emu_gated_linear.argtypes = dims3 + [vp, i64, vp, i64, vp, vp, ci, vp, i64, vp, vp, i64, vp]
        L.sgemm_emu_gated_linear_backward_workspace.argtypes = dims3
        L.sgemm_emu_gated_linear_backward.argtypes = dims3 + [vp, i64, vp, i64, vp, ci, vp, i64, vp, i64, vp, i64,
                                                              vp, vp, i64, vp]
        L.sgemm_emu_adapter_linear_workspace.argtypes = dims3 + [vp, i64, vp, i64, vp, i64, i64, vp, vp]
        L.sgemm_emu_adapter_linear.argtypes = dims3 + [vp, i64, vp, i64, vp, vp, i64, i64, vp, vp, vp, vp, vp, i64,
                                                       vp, vp, i64, vp]
        L.sgemm_emu_adapter_linear_backward_workspace.argtypes = dims3 + [i64, i64]
        L.sgemm_emu_adapter_linear_backward.argtypes = dims3 + [vp, i64, vp, i64, i64, vp, vp, vp, vp, vp, vp, i64,
                                                                vp, i64, vp, vp, vp, i64, vp]
        L.sgemm_emu_few_rows.argtypes = []
        for name in OPS_EXPORTS:
            getattr(L, name).restype = i64 if name.endswith(("_workspace", "_bytes")) else ci
        FEW_ROWS = L.sgemm_emu_few_rows()
        _OPS = L
    return _OPS


def ok(status, where):
    """Raise SgemmEmuError for a negative status or size; else return it."""
    if status < 0:
        raise SgemmEmuError(int(status), where)
    return status


# ---------------------------------------------------------------- tensor arguments

def check_tensor(t, name, dtype, shape):
    """A tensor of `dtype` and `shape` (None: any extent) on the current HIP device."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch tensor, got {type(t).__name__}")
    if t.dtype is not dtype:
        raise TypeError(f"{name}: expected dtype {dtype}, got {t.dtype}")
    have = t.shape
    if len(have) != len(shape) or any([w is not None and s != w for s, w in zip(have, shape)]):
        raise ValueError(f"{name}: expected shape {tuple('any' if w is None else w for w in shape)}, "
                         f"got {tuple(have)}")
    if not t.is_cuda or t.get_device() != torch.cuda.current_device():
        raise ValueError(f"{name}: expected a tensor on the current HIP device, got {t.device}")


def rows_of(t):
    """A 2-D tensor whose rows lie one after another with unit stride along columns (itself, or a
    contiguous copy of a transposed, expanded or overlapping one, or of one whose rows lie further
    apart than the library takes), and its leading dimension.  The stride of a single row means
    nothing."""
    rows, cols = t.shape
    ld, step = t.stride()
    if (cols > 1 and step != 1) or (rows > 1 and not cols <= ld <= MAX_LD):
        t = t.contiguous()
        ld = cols
    return t, ld if rows > 1 and ld > 0 else max(cols, 1)


def forward_mode():
    """Whether a level of forward-mode differentiation is open: operands may then carry tangents, which
    only a call through an autograd function sees (and refuses)."""
    return getattr(forward_ad, "_current_level", 0) >= 0   # torch's own record; without it, as if one were


def scratch(nbytes, like):
    """Workspace of a call on `like`'s device: torch's allocator keeps it in the stream's order."""
    return like.new_empty(nbytes, dtype=torch.uint8) if nbytes else None


# Workspace bytes of a call on few rows by its dimensions (which alone decide them there), so that
# the calls where latency counts ask once.
_FEW_BYTES = {}


def few_bytes(key, query):
    n = _FEW_BYTES.get(key)
    if n is None:
        n = _FEW_BYTES[key] = ok(query(), "workspace query")
    return n


def addr(t):
    return None if t is None else t.data_ptr() or None


def current_stream():
    return torch.cuda.current_stream().cuda_stream


# torch.cuda.current_stream() builds a Stream object (2 us); torch's own accessor gives the handle alone.
_RAW_STREAM = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def stream_of(device_index):
    """The handle of torch's current stream on a device."""
    return _RAW_STREAM(device_index) if _RAW_STREAM is not None else current_stream()


class WeightPlan:
    """A weight laid out for the products (sgemm_emu_plan_weight): `forward` holds W (None where a
    bfloat16 weight is read as it lies), `backward` W^T (None unless asked for).  It holds the
    values of the weight at the time: lay a changed weight out again.  `gated`: laid out for
    gated_linear (gate and up rows alternate), else for adapter_linear."""

    __slots__ = ("dtype", "shape", "device", "gated", "forward", "backward")

    def __init__(self, weight, gated=False, forward=True, backward=False):
        w = weight.detach()
        if w.dtype not in DTYPES:
            raise TypeError(f"weight: expected dtype float32 or bfloat16, got {w.dtype}")
        check_tensor(w, "weight", w.dtype, (None, None))
        w, ld = rows_of(w)
        self.dtype, self.shape, self.device, self.gated = w.dtype, tuple(w.shape), w.device, gated
        # a bfloat16 weight with 16-byte aligned rows needs no layout for the forward product
        lies = w.dtype == torch.bfloat16 and w.shape[1] % 8 == 0 and ld % 8 == 0 and w.data_ptr() % 16 == 0
        rows = SGEMM_EMU_PLAN_GATED if gated else SGEMM_EMU_PLAN_ROWS
        self.forward = self._lay_out(w, ld, rows) if forward and not lies else None
        self.backward = self._lay_out(w, ld, SGEMM_EMU_PLAN_TRANSPOSED) if backward else None

    @staticmethod
    def _lay_out(w, ld, layout):
        L, dt = ops_lib(), DTYPES[w.dtype]
        rows, cols = w.shape
        nbytes = ok(L.sgemm_emu_plan_bytes(dt, rows, cols, layout), "sgemm_emu_plan_bytes")
        plan = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=w.device)
        ok(L.sgemm_emu_plan_weight(dt, rows, cols, addr(w), ld, layout, plan.data_ptr(), current_stream()),
           "sgemm_emu_plan_weight")
        return plan

    def check(self, weight, gated):
        """Raises where this is no layout of such a weight for gated_linear (gated) or adapter_linear.
        The two differ in the order of W's rows, so one never stands in for the other."""
        if self.gated != gated:
            mine, other = ("gated", "adapters") if gated else ("adapters", "gated")
            raise ValueError(f"plan: laid out by {other}.plan_weight, expected one of {mine}.plan_weight")
        if self.dtype != weight.dtype or self.shape != tuple(weight.shape) or self.device != weight.device:
            raise ValueError(f"plan: laid out for a {self.dtype} weight of shape {self.shape} on {self.device}, got "
                             f"{weight.dtype} {tuple(weight.shape)} on {weight.device}")


class FixedWeight:
    """Tells whether a module's weight is still the one that was fixed: the same tensor, with no
    change that torch counts.  A copy of the module (deepcopy, pickle) holds a copy of its weight,
    which is as fixed as the original was.

    A layout (WeightPlan) is not kept with it: writes through `weight.data` count nowhere, and a
    layout kept over them would multiply with the old weight."""

    __slots__ = ("weight", "version")

    def __init__(self, weight):
        self.weight, self.version = weight, _version(weight)

    def check(self, weight):
        if weight is not self.weight or _version(weight) != self.version:
            raise RuntimeError("the weight changed after fix_weights(); call it again")

    def __getstate__(self):
        return self.weight, _version(self.weight) == self.version

    def __setstate__(self, state):
        self.weight, fixed = state
        self.version = _version(self.weight) if fixed else -1


def _version(t):
    """torch's count of a tensor's changes; None for an inference tensor, whose changes it does not count."""
    return None if t.is_inference() else t._version
