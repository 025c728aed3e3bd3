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
from dataclasses import dataclass

from . import (ACT_SILU, DTYPE_BF16, DTYPE_F16, GROUP, PackedWeight, W4A16Error, _act_dtype,
               _dev_ptr, _dtype_code, _PreparedCall, _refuse_grad, _shaped_ptr, _stream_handle, _torch,
               lib)

__all__ = [
    "NORM_NONE", "NORM_RMS", "NORM_LAYER", "Norm", "NormBlockCall", "w4a16_norm_block", "NormGrads",
    "NormBlockBackwardCall", "w4a16_norm_block_backward", "SCORE_SOFTMAX", "SCORE_SIGMOID", "DTYPE_F32",
    "Routing", "RouteCall", "w4a16_route", "RouteBackwardCall", "w4a16_route_backward", "PackedExperts",
    "w4a16_stack_experts", "ExpertsCall", "w4a16_experts", "TransposedExperts", "w4a16_transpose_experts",
    "ExpertsBackwardCall", "w4a16_experts_backward",
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


class ExpertWeightStruct(ctypes.Structure):
    """Mirror of the C struct w4a16_expert_weight."""
    _fields_ = [("Wq", _VP), ("scales", _VP), ("zeros", _VP)]


class ExpertsStruct(ctypes.Structure):
    """Mirror of the C struct w4a16_experts_call."""
    _fields_ = [("X", _VP), ("ids", _VP), ("weights", _VP), ("gate", ExpertWeightStruct),
                ("up", ExpertWeightStruct), ("down", ExpertWeightStruct), ("s", _VP), ("s_down", _VP),
                ("residual", _VP), ("G", _VP), ("U", _VP), ("Y", _VP), ("T", _I64), ("E", _I64), ("k", _I64),
                ("D", _I64), ("N", _I64), ("act", _I32), ("dtype", _I32)]


class ExpertTransposedStruct(ctypes.Structure):
    """Mirror of the C struct w4a16_expert_transposed."""
    _fields_ = [("Wt", _VP), ("meta", _VP)]


class ExpertsBackwardStruct(ctypes.Structure):
    """Mirror of the C struct w4a16_experts_backward_call."""
    _fields_ = [("dY", _VP), ("ids", _VP), ("weights", _VP), ("G", _VP), ("U", _VP),
                ("gate", ExpertTransposedStruct), ("up", ExpertTransposedStruct),
                ("down", ExpertTransposedStruct), ("s", _VP), ("s_down", _VP), ("add", _VP), ("dX", _VP),
                ("dweights", _VP), ("T", _I64), ("E", _I64), ("k", _I64), ("D", _I64), ("N", _I64),
                ("act", _I32), ("dtype", _I32), ("dweights_f32", _I32)]


def _declare(L):
    """Argument types of this module's entry points (called once the library is loaded)."""
    ref, sz, cs, ci = ctypes.POINTER, ctypes.POINTER(ctypes.c_size_t), ctypes.c_size_t, ctypes.c_int
    for name, args in (
            ("w4a16_norm_block", [ref(NormCallStruct), _VP]),
            ("w4a16_norm_block_backward_workspace_size", [ref(NormBackwardStruct), sz]),
            ("w4a16_norm_block_backward", [ref(NormBackwardStruct), _VP, cs, _VP]),
            ("w4a16_route", [ref(RoutingStruct), _VP, _VP, _VP, _VP, _VP]),
            ("w4a16_route_backward", [ref(RoutingStruct), _VP, _VP, _VP, _VP, _VP]),
            ("w4a16_experts_workspace_size", [ref(ExpertsStruct), sz]),
            ("w4a16_experts", [ref(ExpertsStruct), _VP, cs, _VP]),
            ("w4a16_experts_backward_workspace_size", [ref(ExpertsBackwardStruct), sz]),
            ("w4a16_experts_backward", [ref(ExpertsBackwardStruct), _VP, cs, _VP])):
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
    gate_rows = min(gate_rows, max(T, 1))  # (the same gates, and a number of 64 bits)
    if T == 0 and gate.shape[0] == 1:
        return (1, D), gate_rows
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
    _act_dtype(x, "x")
    if y is None and (gate is not None or (post is not None and post.kind != NORM_NONE)):
        raise ValueError("post and gate need y")
    r = x if y is None and alpha == 1.0 else torch.empty_like(x)
    h = torch.empty_like(x) if pre is not None else None
    call = NormBlockCall(x, y, None if r is x else r, h, post, pre, gate, gate_rows, alpha)
    if r is not x or h is not None:
        call()
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
        if T == 0 and g.gate is not None:
            self.function = self._with_zeros(self.function, g.gate, device)

    @staticmethod
    def _with_zeros(function, dgate, device):
        """Of no tokens the C call sees a gate of no rows and writes none: zeros, on the stream it gets."""
        torch = _torch()

        def call(*args):
            rc = function(*args)
            if not rc:
                handle = getattr(args[-1], "value", args[-1]) or 0
                with torch.cuda.stream(torch.cuda.ExternalStream(handle, device)):
                    dgate.zero_()
            return rc
        return call


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


# ---- experts ---------------------------------------------------------------------------------

@dataclass
class PackedExperts:
    """E packed INT4 weights [N][K] of one shape, one after the other in each buffer (the buffers
    of PackedWeight, E times as long)."""
    wq: "object"
    scales: "object"
    zeros: "object"
    E: int
    N: int
    K: int


def w4a16_stack_experts(weights) -> PackedExperts:
    """PackedExperts of a list of PackedWeight (INT4 codes, one shape, no fp16 outliers)."""
    torch = _torch()
    weights = list(weights)
    if not weights:
        raise ValueError("at least one expert")
    first = weights[0]
    for w in weights:
        if (w.N, w.K, w.wbits) != (first.N, first.K, 4):
            raise ValueError("experts must be INT4 weights of one shape")
        if w.outlier_ptrs()[0] is not None:
            raise ValueError("experts take no fp16 outliers")
    return PackedExperts(*(torch.cat([getattr(w, n) for w in weights]) for n in ("wq", "scales", "zeros")),
                         len(weights), first.N, first.K)


def _expert_struct(w, name, shape, device):
    torch = _torch()
    if (w.E, w.N, w.K) != shape:
        raise ValueError(f"{name} must be {shape[0]} experts of [{shape[1]}][{shape[2]}]")
    meta = (w.E * w.N * (-(-(w.K // GROUP) // 4) * 4),)
    return ExpertWeightStruct(
        _shaped_ptr(w.wq, f"{name}.wq", torch.uint8, (w.E * w.N * w.K // 2,), device),
        _shaped_ptr(w.scales, f"{name}.scales", torch.float16, meta, device),
        _shaped_ptr(w.zeros, f"{name}.zeros", torch.float16, meta, device))


def _slots_ptrs(ids, weights, T, device):
    torch = _torch()
    if ids.dim() != 2:
        raise ValueError("ids must be [T][k]")
    k = ids.shape[1]
    return k, (_shaped_ptr(ids, "ids", torch.int32, (T, k), device),
               _shaped_ptr(weights, "weights", torch.float32, (T, k), device))


class ExpertsCall(_PreparedCall):
    """A prepared w4a16_experts call: Y = residual + the weighted sum of each token's experts,
    act(G) * U through down, G and U the products of X * s with gate and up.

    X, Y and residual (or None; may be Y) [T][D] are fp16 or bf16; ids int32 and weights fp32
    [T][k] as w4a16_route gives them (an id outside 0..E-1: the slot adds nothing); gate, up
    [N][D] and down [D][N] PackedExperts; s fp16 [D] and s_down fp16 [E][N] or None; preact: a
    pair of [T][k][N] tensors that receive G and U, or None."""

    def __init__(self, X, ids, weights, gate, up, down, Y, s=None, s_down=None, act=ACT_SILU, residual=None,
                 preact=None, stream=None, workspace=None):
        torch = _torch()
        dt, device = _act_dtype(X, "X"), X.device
        if X.dim() != 2:
            raise ValueError("X must be [T][D]")
        (T, D), E, N = X.shape, gate.E, gate.N
        k, slots = _slots_ptrs(ids, weights, T, device)
        G, U = preact if preact is not None else (None, None)
        self.keep = (X, ids, weights, gate, up, down, Y, s, s_down, residual, G, U)
        self.call = ExpertsStruct(
            _dev_ptr(X, "X", dt), *slots, _expert_struct(gate, "gate", (E, N, D), device),
            _expert_struct(up, "up", (E, N, D), device), _expert_struct(down, "down", (E, D, N), device),
            _shaped_ptr(s, "s", torch.float16, (D,), device),
            _shaped_ptr(s_down, "s_down", torch.float16, (E, N), device),
            _shaped_ptr(residual, "residual", dt, (T, D), device),
            _shaped_ptr(G, "preact[0]", dt, (T, k, N), device), _shaped_ptr(U, "preact[1]", dt, (T, k, N), device),
            _shaped_ptr(Y, "Y", dt, (T, D), device), T, E, k, D, N, act, _dtype_code(dt))
        nbytes = self._size("w4a16_experts_workspace_size", ctypes.byref(self.call))
        self._prepare(device, nbytes, workspace, stream)
        self._bind("w4a16_experts", ctypes.byref(self.call))


def w4a16_experts(X, ids, weights, gate, up, down, s=None, s_down=None, act=ACT_SILU, residual=None, out=None,
                  preact=None):
    """The weighted sum of each token's experts on the current stream.  Arguments as for
    ExpertsCall."""
    if out is None:
        out = _torch().empty_like(X)
    ExpertsCall(X, ids, weights, gate, up, down, out, s, s_down, act, residual, preact)()
    return out


@dataclass
class TransposedExperts:
    """Transposed copies of PackedExperts for the backward pass, one expert after the other in
    each buffer (layout: w4a16_transpose in include/w4a16.h)."""
    wt: "object"
    meta: "object"
    E: int
    N: int
    K: int


def w4a16_transpose_experts(w: PackedExperts) -> TransposedExperts:
    """The transposed copies that w4a16_experts_backward reads, made once per weight (on the
    current stream)."""
    torch = _torch()
    a, b = ctypes.c_size_t(), ctypes.c_size_t()
    rc = lib().w4a16_transposed_sizes(w.N, w.K, 4, ctypes.byref(a), ctypes.byref(b))
    if rc:
        raise W4A16Error(rc, "w4a16_transposed_sizes")
    dev = w.wq.device
    src = _expert_struct(w, "experts", (w.E, w.N, w.K), dev)
    out = TransposedExperts(torch.empty(w.E * a.value, dtype=torch.uint8, device=dev),
                            torch.empty(w.E * b.value, dtype=torch.uint8, device=dev), w.E, w.N, w.K)
    codes, meta = w.N * w.K // 2, w.N * (-(-(w.K // GROUP) // 4) * 4) * 2
    with torch.cuda.device(dev):
        for e in range(w.E):
            rc = lib().w4a16_transpose(src.Wq + e * codes, src.scales + e * meta, src.zeros + e * meta, w.N, w.K,
                                       4, out.wt.data_ptr() + e * a.value, out.meta.data_ptr() + e * b.value,
                                       _stream_handle(dev))
            if rc:
                raise W4A16Error(rc, "w4a16_transpose")
    return out


def _transposed_struct(w, name, shape, device):
    torch = _torch()
    if (w.E, w.N, w.K) != shape:
        raise ValueError(f"{name} must be {shape[0]} transposed experts of [{shape[1]}][{shape[2]}]")
    rows = -(-w.N // GROUP)
    return ExpertTransposedStruct(
        _shaped_ptr(w.wt, f"{name}.wt", torch.uint8, (w.E * rows * GROUP * w.K // 2,), device),
        _shaped_ptr(w.meta, f"{name}.meta", torch.uint8, (w.E * rows * (w.K // GROUP) * 512,), device))


class ExpertsBackwardCall(_PreparedCall):
    """A prepared w4a16_experts_backward call: dX [T][D] (or None), of the activations' type, and
    dweights [T][k] (or None), fp32 (as w4a16_route_backward takes them) or of that type, from dY,
    the routing and the G and U of the forward; gate, up and down TransposedExperts; add [T][D]
    (or None; may be dX) is added to dX."""

    def __init__(self, dY, ids, weights, G, U, gate, up, down, dX, dweights, s=None, s_down=None, act=ACT_SILU,
                 add=None, stream=None, workspace=None):
        torch = _torch()
        dt, device = _act_dtype(dY, "dY"), dY.device
        if dY.dim() != 2:
            raise ValueError("dY must be [T][D]")
        (T, D), E, N = dY.shape, gate.E, gate.N
        k, slots = _slots_ptrs(ids, weights, T, device)
        self.keep = (dY, ids, weights, G, U, gate, up, down, dX, dweights, s, s_down, add)
        f32 = dweights is not None and dweights.dtype == torch.float32
        self.call = ExpertsBackwardStruct(
            _dev_ptr(dY, "dY", dt), *slots, _shaped_ptr(G, "G", dt, (T, k, N), device),
            _shaped_ptr(U, "U", dt, (T, k, N), device), _transposed_struct(gate, "gate", (E, N, D), device),
            _transposed_struct(up, "up", (E, N, D), device), _transposed_struct(down, "down", (E, D, N), device),
            _shaped_ptr(s, "s", torch.float16, (D,), device),
            _shaped_ptr(s_down, "s_down", torch.float16, (E, N), device),
            _shaped_ptr(add, "add", dt, (T, D), device), _shaped_ptr(dX, "dX", dt, (T, D), device),
            _shaped_ptr(dweights, "dweights", torch.float32 if f32 else dt, (T, k), device), T, E, k, D, N, act,
            _dtype_code(dt), int(f32))
        nbytes = self._size("w4a16_experts_backward_workspace_size", ctypes.byref(self.call))
        self._prepare(device, nbytes, workspace, stream)
        self._bind("w4a16_experts_backward", ctypes.byref(self.call))


def w4a16_experts_backward(dY, ids, weights, G, U, gate, up, down, s=None, s_down=None, act=ACT_SILU, add=None):
    """Backward of w4a16_experts on the current stream: (dX, dweights), dweights fp32.  Arguments
    as for ExpertsBackwardCall."""
    torch = _torch()
    dX, dw = torch.empty_like(dY), torch.empty(ids.shape, dtype=torch.float32, device=dY.device)
    ExpertsBackwardCall(dY, ids, weights, G, U, gate, up, down, dX, dw, s, s_down, act, add)()
    return dX, dw
