"""The expert feed-forward block: norms before and after the block with its gate and residual
scale, routing of tokens to experts, and the experts' products over packed INT4 weights, with
their backward passes.  The C ABI is in include/w4a16.h; this module marshals arguments, as the
rest of the package does.

    r, h = w4a16_norm_block(x, y, post=Norm(NORM_RMS, w1), pre=Norm(NORM_RMS, w2))
    ids, weights = w4a16_route(router_logits, Routing(k=8))
    y = w4a16_experts(h, ids, weights, gate, up, down)      # PackedExperts each
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass, field

from . import (ACT_SILU, DTYPE_BF16, DTYPE_F16, GROUP, PackedWeight, W4A16Error, _act_dtype,
               _dev_ptr, _dtype_code, _PreparedCall, _refuse_grad, _shaped_ptr, _stream_handle, _torch,
               lib)

__all__ = [
    "NORM_NONE", "NORM_RMS", "NORM_LAYER", "Norm", "NormBlockCall", "w4a16_norm_block", "NormGrads",
    "NormBlockBackwardCall", "w4a16_norm_block_backward", "SCORE_SOFTMAX", "SCORE_SIGMOID", "DTYPE_F32",
    "Routing", "RouteCall", "w4a16_route", "RouteBackwardCall", "w4a16_route_backward",
]

NORM_NONE, NORM_RMS, NORM_LAYER = 0, 1, 2
SCORE_SOFTMAX, SCORE_SIGMOID = 0, 1
DTYPE_F32 = 2

_VP, _I64, _I32, _F32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float


class NormStruct(ctypes.Structure):
    """Mirror of the C struct w4a16_norm."""
    _fields_ = [("weight", _VP), ("bias", _VP), ("eps", _F32), ("kind", _I32)]


class NormCallStruct(ctypes.Structure):
    """Mirror of the C struct w4a16_norm_call."""
    _fields_ = [("x", _VP), ("y", _VP), ("gate", _VP), ("post", NormStruct), ("pre", NormStruct),
                ("r", _VP), ("h", _VP), ("T", _I64), ("D", _I64), ("gate_rows", _I64),
                ("alpha", _F32), ("dtype", _I32)]


class NormBackwardStruct(ctypes.Structure):
    """Mirror of the C struct w4a16_norm_backward_call."""
    _fields_ = [("dr", _VP), ("dh", _VP), ("y", _VP), ("r", _VP), ("gate", _VP),
                ("post", NormStruct), ("pre", NormStruct), ("dx", _VP), ("dy", _VP), ("dgate", _VP),
                ("dpost_weight", _VP), ("dpost_bias", _VP), ("dpre_weight", _VP),
                ("dpre_bias", _VP), ("T", _I64), ("D", _I64), ("gate_rows", _I64), ("alpha", _F32),
                ("dtype", _I32)]


class RoutingStruct(ctypes.Structure):
    """Mirror of the C struct w4a16_routing."""
    _fields_ = [("T", _I64), ("E", _I64), ("k", _I64), ("score", _I32), ("groups", _I32),
                ("topk_groups", _I32), ("renormalize", _I32), ("scale", _F32), ("dtype", _I32)]


def _declare(L):
    """Argument types of this module's entry points (called once the library is loaded)."""
    ref, sz, cs, ci = ctypes.POINTER, ctypes.POINTER(ctypes.c_size_t), ctypes.c_size_t, ctypes.c_int
    for name, args in (
            ("w4a16_norm_block", [ref(NormCallStruct), _VP]),
            ("w4a16_norm_block_backward_workspace_size", [ref(NormBackwardStruct), sz]),
            ("w4a16_norm_block_backward", [ref(NormBackwardStruct), _VP, cs, _VP]),
            ("w4a16_route", [ref(RoutingStruct), _VP, _VP, _VP, _VP, _VP]),
            ("w4a16_route_backward", [ref(RoutingStruct), _VP, _VP, _VP, _VP, _VP])):
        getattr(L, name).argtypes = args
        getattr(L, name).restype = ci


class _PlainCall(_PreparedCall):
    """A prepared call of an entry point that takes no workspace."""

    def _bind_plain(self, name, device, stream, *args):
        self._prepare(device, 0, None, stream)
        self._bind(name)
        self.args = args


# ---- norms ---------------------------------------------------------------------------------

@dataclass
class Norm:
    """A norm over the columns of a row: NORM_RMS or NORM_LAYER, weight and bias [D] of the
    activations' type (None: 1 and 0)."""
    kind: int = NORM_RMS
    weight: "object" = None
    bias: "object" = None
    eps: float = 1e-6


def _norm_struct(norm, name, dt, D, device):
    if norm is None:
        return NormStruct(None, None, 0.0, NORM_NONE)
    return NormStruct(_shaped_ptr(norm.weight, f"{name}.weight", dt, (D,), device),
                      _shaped_ptr(norm.bias, f"{name}.bias", dt, (D,), device), norm.eps, norm.kind)


def _gate_shape(gate, gate_rows, T, D):
    """(shape, gate_rows) of the gate of T tokens; a gate of one row serves all of them."""
    if gate is None:
        return None, 0
    if gate.dim() == 1:
        return (D,), max(T, 1)
    if gate_rows is None:
        if gate.shape[0] not in (1, T):
            raise ValueError("gate_rows must be given for a gate that is neither one row nor one per token")
        gate_rows = max(T, 1) if gate.shape[0] == 1 else 1
    if gate_rows < 1:
        raise ValueError("gate_rows must be at least 1")
    return (-(-T // gate_rows), D), gate_rows


class NormBlockCall(_PlainCall):
    """A prepared w4a16_norm_block call: r = alpha * x + gate * post(y), h = pre(r).

    x, r, h [T][D] and y [T][D] (or None) are fp16 or bf16; post and pre are Norm or None;
    gate is [D], or [ceil(T / gate_rows)][D] with row t // gate_rows for token t.  r may be None;
    h is None exactly where pre is.  r and h may each be x or y."""

    def __init__(self, x, y, r, h, post=None, pre=None, gate=None, gate_rows=None, alpha=1.0, stream=None):
        dt, device = _act_dtype(x, "x"), x.device
        if x.dim() != 2:
            raise ValueError("x must be [T][D]")
        T, D = x.shape
        self.keep = (x, y, r, h, post, pre, gate)
        shape, rows = _gate_shape(gate, gate_rows, T, D)
        self.call = NormCallStruct(
            _dev_ptr(x, "x", dt), _shaped_ptr(y, "y", dt, (T, D), device),
            _shaped_ptr(gate, "gate", dt, shape, device), _norm_struct(post, "post", dt, D, device),
            _norm_struct(pre, "pre", dt, D, device), _shaped_ptr(r, "r", dt, (T, D), device),
            _shaped_ptr(h, "h", dt, (T, D), device), T, D, rows, alpha, _dtype_code(dt))
        self._bind_plain("w4a16_norm_block", device, stream, ctypes.byref(self.call))


def w4a16_norm_block(x, y=None, post=None, pre=None, gate=None, gate_rows=None, alpha=1.0):
    """(r, h) = (alpha * x + gate * post(y), pre(r)) on the current stream; h is None without
    pre, and r is x itself where y is None and alpha is 1.  Arguments as for NormBlockCall."""
    torch = _torch()
    r = x if y is None and alpha == 1.0 else torch.empty_like(x)
    h = torch.empty_like(x) if pre is not None else None
    if r is not x or h is not None:
        NormBlockCall(x, y, None if r is x else r, h, post, pre, gate, gate_rows, alpha)()
    return r, h


@dataclass
class NormGrads:
    """The fp32 gradients that a backward call writes, each a tensor or None: gate (the gate's
    shape) and the norms' weights and biases [D]."""
    gate: "object" = None
    post_weight: "object" = None
    post_bias: "object" = None
    pre_weight: "object" = None
    pre_bias: "object" = None


class NormBlockBackwardCall(_PreparedCall):
    """A prepared w4a16_norm_block_backward call: dx, dy [T][D] (each or None) and the gradients in
    `grads`, from dr (the gradient of r from elsewhere, or None), dh (required exactly where pre
    is given) and the forward's y and r."""

    def __init__(self, dr, dh, y, r, dx, dy, grads=None, post=None, pre=None, gate=None, gate_rows=None,
                 alpha=1.0, stream=None, workspace=None):
        torch = _torch()
        first = dh if dr is None else dr
        if first is None:
            raise ValueError("dr or dh must be given")
        dt, device = _act_dtype(first, "dr" if dr is not None else "dh"), first.device
        if first.dim() != 2:
            raise ValueError("dr and dh must be [T][D]")
        T, D = first.shape
        g = grads or NormGrads()
        self.keep = (dr, dh, y, r, dx, dy, g.gate, g.post_weight, g.post_bias, g.pre_weight, g.pre_bias,
                     post, pre, gate)
        shape, rows = _gate_shape(gate, gate_rows, T, D)
        if g.gate is not None and gate is None:
            raise ValueError("a gradient of the gate needs the gate")

        def rows_ptr(t, name):
            return _shaped_ptr(t, name, dt, (T, D), device)

        def grad_ptr(t, name, s=(D,)):
            return _shaped_ptr(t, name, torch.float32, s, device)

        self.call = NormBackwardStruct(
            rows_ptr(dr, "dr"), rows_ptr(dh, "dh"), rows_ptr(y, "y"), rows_ptr(r, "r"),
            _shaped_ptr(gate, "gate", dt, shape, device), _norm_struct(post, "post", dt, D, device),
            _norm_struct(pre, "pre", dt, D, device), rows_ptr(dx, "dx"), rows_ptr(dy, "dy"),
            grad_ptr(g.gate, "grads.gate", shape), grad_ptr(g.post_weight, "grads.post_weight"),
            grad_ptr(g.post_bias, "grads.post_bias"), grad_ptr(g.pre_weight, "grads.pre_weight"),
            grad_ptr(g.pre_bias, "grads.pre_bias"), T, D, rows, alpha, _dtype_code(dt))
        nbytes = self._size("w4a16_norm_block_backward_workspace_size", ctypes.byref(self.call))
        self._prepare(device, nbytes, workspace, stream)
        self._bind("w4a16_norm_block_backward", ctypes.byref(self.call))


def w4a16_norm_block_backward(dr, dh, y=None, r=None, post=None, pre=None, gate=None, gate_rows=None,
                              alpha=1.0):
    """Backward of w4a16_norm_block on the current stream: (dx, dy, NormGrads), with the
    gradients of every weight, bias and gate that is given.  dy is None where y is."""
    torch = _torch()
    first = dh if dr is None else dr
    if first is None:
        raise ValueError("dr or dh must be given")

    def like(t):
        return None if t is None else torch.empty(t.shape, dtype=torch.float32, device=t.device)

    grads = NormGrads(like(gate), *(like(t) for n in (post, pre)
                                    for t in ((n.weight, n.bias) if n is not None else (None, None))))
    dx, dy = torch.empty_like(first), None if y is None else torch.empty_like(first)
    NormBlockBackwardCall(dr, dh, y, r, dx, dy, grads, post, pre, gate, gate_rows, alpha)()
    return dx, dy, grads


# ---- routing ---------------------------------------------------------------------------------

@dataclass
class Routing:
    """How tokens choose their experts (w4a16_route in include/w4a16.h): the k best of
    score + bias, within the topk_groups best of `groups` groups; weights scale * score,
    renormalised over the chosen experts or not."""
    k: int
    score: int = SCORE_SOFTMAX
    groups: int = 1
    topk_groups: int = 1
    renormalize: bool = True
    scale: float = 1.0


def _logit_dtype(t):
    torch = _torch()
    codes = {torch.float16: DTYPE_F16, torch.bfloat16: DTYPE_BF16, torch.float32: DTYPE_F32}
    if not isinstance(t, torch.Tensor) or t.dtype not in codes:
        raise TypeError("logits must be a float16, bfloat16 or float32 tensor")
    if t.dim() != 2:
        raise ValueError("logits must be [T][E]")
    _refuse_grad(t, "logits")
    return codes[t.dtype]


def _routing_struct(routing, logits):
    code = _logit_dtype(logits)
    return RoutingStruct(logits.shape[0], logits.shape[1], routing.k, routing.score, routing.groups,
                         routing.topk_groups, int(bool(routing.renormalize)), routing.scale, code)


class RouteCall(_PlainCall):
    """A prepared w4a16_route call: logits [T][E] (fp16, bf16 or fp32), bias fp32 [E] or None (it
    goes into the choice alone); writes ids int32 [T][k] and weights fp32 [T][k]."""

    def __init__(self, logits, routing, ids, weights, bias=None, stream=None):
        torch = _torch()
        self.routing = _routing_struct(routing, logits)
        T, E = logits.shape
        device = logits.device
        self.keep = (logits, ids, weights, bias)
        self._bind_plain(
            "w4a16_route", device, stream, ctypes.byref(self.routing),
            _dev_ptr(logits, "logits", logits.dtype), _shaped_ptr(bias, "bias", torch.float32, (E,), device),
            _shaped_ptr(ids, "ids", torch.int32, (T, routing.k), device),
            _shaped_ptr(weights, "weights", torch.float32, (T, routing.k), device))


def w4a16_route(logits, routing, bias=None):
    """(ids, weights) of each token's experts on the current stream.  Arguments as for RouteCall."""
    torch = _torch()
    _logit_dtype(logits)
    shape = (logits.shape[0], routing.k)
    ids = torch.empty(shape, dtype=torch.int32, device=logits.device)
    weights = torch.empty(shape, dtype=torch.float32, device=logits.device)
    RouteCall(logits, routing, ids, weights, bias)()
    return ids, weights


class RouteBackwardCall(_PlainCall):
    """A prepared w4a16_route_backward call: dlogits [T][E] of the logits' type from dweights fp32
    [T][k], the logits and the ids of the forward."""

    def __init__(self, dweights, logits, ids, routing, dlogits, stream=None):
        torch = _torch()
        self.routing = _routing_struct(routing, logits)
        device, slots = logits.device, (logits.shape[0], routing.k)
        self.keep = (dweights, logits, ids, dlogits)
        self._bind_plain(
            "w4a16_route_backward", device, stream, ctypes.byref(self.routing),
            _shaped_ptr(dweights, "dweights", torch.float32, slots, device),
            _dev_ptr(logits, "logits", logits.dtype),
            _shaped_ptr(ids, "ids", torch.int32, slots, device),
            _shaped_ptr(dlogits, "dlogits", logits.dtype, logits.shape, device))


def w4a16_route_backward(dweights, logits, ids, routing):
    """Gradient of the logits on the current stream.  Arguments as for RouteBackwardCall."""
    dlogits = _torch().empty_like(logits)
    RouteBackwardCall(dweights, logits, ids, routing, dlogits)()
    return dlogits
