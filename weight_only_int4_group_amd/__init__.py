"""Weight-only INT4 per-group quantization (W4A16) for AMD Instinct MI355X.

Thin ctypes binding over ``libw4a16.so`` (C ABI in ``include/w4a16.h``).  The
binding only marshals arguments: it checks tensor dtypes/devices, allocates
outputs with torch (device memory and streams are torch's), and passes raw
pointers and the current HIP stream to the library.  Every step of the
computation runs in the library's HIP kernels; there is no fallback.

    from weight_only_int4_group_amd import w4a16_quantize_pack, w4a16_gemm
    pw = w4a16_quantize_pack(W, s)        # W: fp16 [N][K] cuda, s: fp16 [K] or None
    Y = w4a16_gemm(X, pw, s)              # X: fp16 [M][K] cuda -> Y: fp16 [M][N]
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass

from .build import LIB_PATH as _BUILT_LIB

# the in-tree build; W4A16_LIB names another build of the same sources (the
# host-sanitized one, for CPU runs of the validation tests)
LIB_PATH = os.environ.get("W4A16_LIB") or _BUILT_LIB

__all__ = [
    "W4A16Error", "PackedWeight", "GROUP", "PATH_AUTO", "PATH_SKINNY", "PATH_TILED",
    "PATH_SKINNY_WINDOW", "QUANT_ASYM", "QUANT_SYM", "QUANT_ASYM_CHANNEL", "QUANT_ASYM_TENSOR",
    "QUANT_ASYM8",
    "lib",
    "w4a16_packed_sizes", "w4a16_quantize_pack", "w4a16_gemm", "w4a16_gemm_path",
    "w4a16_select_path", "w4a16_strerror", "w4a16_version", "EXPORTED_SYMBOLS",
    "w4a16_gemm_grouped", "GroupedCall", "w4a16_spec_verify",
    "w4a16_spec_verify_workspace_size", "SpecVerifyCall", "w4a16_quantize_pack_outliers",
    "w4a16_outlier_workspace_size", "page_outlier_count", "DTYPE_F16", "DTYPE_BF16",
    "w4a16_quantize_pack_gptq", "w4a16_gemm_grouped_static", "STATIC_SCRATCH_BYTES",
    "SHARED_SCRATCH_BYTES",
    "ACT_NONE", "ACT_RELU", "ACT_SILU", "ACT_GELU", "ACT_GELU_TANH", "Epilogue", "LinearCall",
    "w4a16_linear", "GatedCall", "w4a16_gated", "TransposedWeight", "w4a16_transpose",
    "BackwardTerm", "LinearBackwardCall", "w4a16_linear_backward", "GatedBackwardCall",
    "w4a16_gated_backward",
]

GROUP = 128
PATH_AUTO, PATH_SKINNY, PATH_TILED, PATH_SKINNY_WINDOW = 0, 1, 2, 3
QUANT_ASYM, QUANT_SYM, QUANT_ASYM_CHANNEL, QUANT_ASYM_TENSOR, QUANT_ASYM8 = 0, 1, 2, 3, 4
DTYPE_F16, DTYPE_BF16 = 0, 1
ACT_NONE, ACT_RELU, ACT_SILU, ACT_GELU, ACT_GELU_TANH = 0, 1, 2, 3, 4
STATUS = {0: "W4A16_OK", -1: "W4A16_EINVAL", -2: "W4A16_EALIGN", -3: "W4A16_EUNSUPPORTED",
          -4: "W4A16_ENONFINITE", -5: "W4A16_ERANGE", -6: "W4A16_EHIP", -7: "W4A16_ESCRATCH"}
STATIC_SCRATCH_BYTES = 64 << 20   # W4A16_STATIC_SCRATCH_BYTES
SHARED_SCRATCH_BYTES = 32 << 20   # W4A16_SHARED_SCRATCH_BYTES
EXPORTED_SYMBOLS = ("w4a16_packed_sizes", "w4a16_packed_sizes_mode", "w4a16_quantize_pack",
                    "w4a16_quantize_pack_mode",
                    "w4a16_gemm",
                    "w4a16_gemm_path", "w4a16_gemm_grouped", "w4a16_gemm_grouped_ws",
                    "w4a16_gemm_grouped_static",
                    "w4a16_gemm_workspace_size", "w4a16_outlier_workspace_size",
                    "w4a16_gptq_workspace_size", "w4a16_quantize_pack_gptq",
                    "w4a16_quantize_pack_outliers", "w4a16_spec_verify",
                    "w4a16_spec_verify_workspace_size", "w4a16_select_path",
                    "w4a16_strerror", "w4a16_version",
                    "w4a16_linear", "w4a16_linear_workspace_size", "w4a16_gated",
                    "w4a16_gated_workspace_size", "w4a16_transposed_sizes", "w4a16_transpose",
                    "w4a16_linear_backward", "w4a16_linear_backward_workspace_size",
                    "w4a16_gated_backward", "w4a16_gated_backward_workspace_size",
                    "w4a16_norm_block", "w4a16_norm_block_backward_workspace_size",
                    "w4a16_norm_block_backward", "w4a16_route", "w4a16_route_backward",
                    "w4a16_experts_workspace_size", "w4a16_experts",
                    "w4a16_experts_backward_workspace_size", "w4a16_experts_backward")


class Problem(ctypes.Structure):
    """Mirror of the C struct w4a16_problem."""
    _fields_ = [("X", ctypes.c_void_p), ("Wq", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("zeros", ctypes.c_void_p), ("s", ctypes.c_void_p), ("Y", ctypes.c_void_p),
                ("M", ctypes.c_int64), ("N", ctypes.c_int64), ("K", ctypes.c_int64),
                ("o_row_ptr", ctypes.c_void_p), ("o_col", ctypes.c_void_p),
                ("o_val", ctypes.c_void_p), ("dtype", ctypes.c_int32), ("wbits", ctypes.c_int32)]


class EpilogueStruct(ctypes.Structure):
    """Mirror of the C struct w4a16_epilogue."""
    _fields_ = [("bias", ctypes.c_void_p), ("residual", ctypes.c_void_p),
                ("preact", ctypes.c_void_p), ("act", ctypes.c_int32)]


class BackwardTermStruct(ctypes.Structure):
    """Mirror of the C struct w4a16_backward_term."""
    _fields_ = [("dY", ctypes.c_void_p), ("preact", ctypes.c_void_p), ("dZ", ctypes.c_void_p),
                ("dbias", ctypes.c_void_p), ("Wt", ctypes.c_void_p), ("meta", ctypes.c_void_p),
                ("N", ctypes.c_int64), ("act", ctypes.c_int32), ("wbits", ctypes.c_int32)]


class W4A16Error(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {STATUS.get(status, status)} ({w4a16_strerror(status)})")


_lib = None


def lib() -> ctypes.CDLL:
    """Load libw4a16.so (built in-tree by ``weight_only_int4_group_amd.build``)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                           "`python -m weight_only_int4_group_amd.build` (needs hipcc)")
    L = ctypes.CDLL(LIB_PATH)
    i64, vp, sz = ctypes.c_int64, ctypes.c_void_p, ctypes.POINTER(ctypes.c_size_t)
    L.w4a16_packed_sizes.argtypes = [i64, i64, sz, sz, sz]
    L.w4a16_packed_sizes_mode.argtypes = [i64, i64, ctypes.c_int, sz, sz, sz]
    L.w4a16_quantize_pack.argtypes = [vp, vp, i64, i64, vp, vp, vp, vp]
    L.w4a16_quantize_pack_mode.argtypes = [vp, vp, i64, i64, ctypes.c_int, vp, vp, vp, vp]
    L.w4a16_gemm.argtypes = [vp, vp, vp, vp, vp, vp, i64, i64, i64, vp]
    L.w4a16_gemm_path.argtypes = [vp, vp, vp, vp, vp, vp, i64, i64, i64, ctypes.c_int, vp]
    L.w4a16_gemm_grouped.argtypes = [ctypes.POINTER(Problem), ctypes.c_int, vp]
    L.w4a16_gemm_grouped_ws.argtypes = [ctypes.POINTER(Problem), ctypes.c_int, vp,
                                        ctypes.c_size_t, vp]
    L.w4a16_gemm_workspace_size.argtypes = [ctypes.POINTER(Problem), ctypes.c_int, sz]
    L.w4a16_gemm_grouped_static.argtypes = [ctypes.POINTER(Problem), ctypes.c_int, vp]
    L.w4a16_spec_verify.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, vp, ctypes.c_size_t, vp,
                                    vp, vp]
    L.w4a16_spec_verify_workspace_size.argtypes = [i64, i64, i64, ctypes.POINTER(ctypes.c_size_t)]
    L.w4a16_outlier_workspace_size.argtypes = [i64, i64, sz]
    L.w4a16_quantize_pack_outliers.argtypes = [vp, vp, i64, i64, ctypes.c_int, i64, vp, vp, vp,
                                               vp, vp, vp, vp, ctypes.c_size_t, vp]
    L.w4a16_gptq_workspace_size.argtypes = [i64, i64, i64, sz]
    L.w4a16_quantize_pack_gptq.argtypes = [vp, vp, i64, i64, vp, i64, ctypes.c_double, vp, vp, vp,
                                           vp, ctypes.c_size_t, vp]
    pp, ep, bp = (ctypes.POINTER(Problem), ctypes.POINTER(EpilogueStruct),
                  ctypes.POINTER(BackwardTermStruct))
    ci, cs = ctypes.c_int, ctypes.c_size_t
    L.w4a16_linear_workspace_size.argtypes = [pp, ep, ci, sz]
    L.w4a16_linear.argtypes = [pp, ep, ci, vp, cs, vp]
    L.w4a16_gated_workspace_size.argtypes = [pp, pp, sz]
    L.w4a16_gated.argtypes = [pp, pp, vp, vp, ci, vp, vp, cs, vp]
    L.w4a16_transposed_sizes.argtypes = [i64, i64, ci, sz, sz]
    L.w4a16_transpose.argtypes = [vp, vp, vp, i64, i64, ci, vp, vp, vp]
    L.w4a16_linear_backward_workspace_size.argtypes = [bp, ci, i64, i64, ci, sz]
    L.w4a16_linear_backward.argtypes = [bp, ci, vp, vp, vp, i64, i64, ci, vp, cs, vp]
    L.w4a16_gated_backward_workspace_size.argtypes = [bp, bp, i64, i64, ci, sz]
    L.w4a16_gated_backward.argtypes = [vp, bp, bp, vp, vp, vp, i64, i64, ci, vp, cs, vp]
    L.w4a16_select_path.argtypes = [i64, i64, i64]
    L.w4a16_strerror.argtypes = [ctypes.c_int]
    L.w4a16_strerror.restype = ctypes.c_char_p
    L.w4a16_version.argtypes = []
    for name in ("w4a16_packed_sizes", "w4a16_packed_sizes_mode", "w4a16_quantize_pack",
                 "w4a16_quantize_pack_mode",
                 "w4a16_gemm", "w4a16_gemm_path",
                 "w4a16_gemm_grouped", "w4a16_gemm_grouped_ws", "w4a16_gemm_workspace_size",
                 "w4a16_gemm_grouped_static",
                 "w4a16_spec_verify", "w4a16_spec_verify_workspace_size", "w4a16_select_path",
                 "w4a16_outlier_workspace_size", "w4a16_quantize_pack_outliers",
                 "w4a16_gptq_workspace_size", "w4a16_quantize_pack_gptq",
                 "w4a16_linear_workspace_size", "w4a16_linear", "w4a16_gated_workspace_size",
                 "w4a16_gated", "w4a16_transposed_sizes", "w4a16_transpose",
                 "w4a16_linear_backward_workspace_size", "w4a16_linear_backward",
                 "w4a16_gated_backward_workspace_size", "w4a16_gated_backward",
                 "w4a16_version"):
        getattr(L, name).restype = ctypes.c_int
    experts._declare(L)
    _lib = L
    return L


def w4a16_strerror(status: int) -> str:
    return lib().w4a16_strerror(status).decode()


def w4a16_version() -> int:
    return lib().w4a16_version()


def w4a16_packed_sizes(N: int, K: int, mode: int = QUANT_ASYM) -> tuple:
    a, b, c = ctypes.c_size_t(), ctypes.c_size_t(), ctypes.c_size_t()
    rc = lib().w4a16_packed_sizes_mode(N, K, mode, ctypes.byref(a), ctypes.byref(b),
                                       ctypes.byref(c))
    if rc:
        raise W4A16Error(rc, "w4a16_packed_sizes")
    return a.value, b.value, c.value


def w4a16_select_path(M: int, N: int, K: int) -> int:
    return lib().w4a16_select_path(M, N, K)


@dataclass
class PackedWeight:
    """Packed weight: INT4 codes (uint8, N*K/2 bytes) or, with wbits = 8, INT8 codes (N*K
    bytes), and the fp16 scale and zero-point buffers (flat, in the 4-group-quad layout
    of include/w4a16.h); with fp16 outliers
    (w4a16_quantize_pack_outliers) also their row pointers (int32 [N+1]), columns
    (int32) and values (fp16)."""
    wq: "object"
    scales: "object"
    zeros: "object"
    N: int
    K: int
    o_row_ptr: "object" = None
    o_col: "object" = None
    o_val: "object" = None
    wbits: int = 4      # 8: INT8 codes (QUANT_ASYM8)

    def outlier_ptrs(self):
        """(row_ptr, col, val) device pointers, or three None without outliers."""
        if self.o_row_ptr is None or self.o_col is None or self.o_col.numel() == 0:
            return None, None, None
        torch = _torch()
        return (_dev_ptr(self.o_row_ptr, "o_row_ptr", torch.int32, self.N + 1),
                _dev_ptr(self.o_col, "o_col", torch.int32),
                _dev_ptr(self.o_val, "o_val", torch.float16, self.o_col.numel()))


def _torch():
    import torch
    return torch


def _stream_handle(dev):
    return ctypes.c_void_p(_torch().cuda.current_stream(dev).cuda_stream)


def _dev_ptr(t, name, dtype=None, numel=None):
    torch = _torch()
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a device (cuda) tensor")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if numel is not None and t.numel() != numel:
        raise ValueError(f"{name} must have {numel} elements, got {t.numel()}")
    return ctypes.c_void_p(t.data_ptr())


def w4a16_quantize_pack(W, s=None, out: PackedWeight | None = None,
                        mode: int = QUANT_ASYM) -> PackedWeight:
    """Quantize fp16 W[N][K] (AWQ scale s[K] or None) into a PackedWeight (blocks).
    mode: QUANT_ASYM (w4a16_quantize_pack), QUANT_SYM (signed -7..7 grid),
    QUANT_ASYM_CHANNEL or QUANT_ASYM_TENSOR (one scale per row or per tensor), or
    QUANT_ASYM8 (INT8 codes, one byte per weight)."""
    torch = _torch()
    if W.dim() != 2:
        raise ValueError("W must be 2-D [N][K]")
    N, K = W.shape
    wq_b, sc_b, z_b = w4a16_packed_sizes(N, K, mode)
    if out is None:
        out = PackedWeight(torch.empty(wq_b, dtype=torch.uint8, device=W.device),
                           torch.empty(sc_b // 2, dtype=torch.float16, device=W.device),
                           torch.empty(z_b // 2, dtype=torch.float16, device=W.device),
                           N, K, wbits=8 if mode == QUANT_ASYM8 else 4)
    rc = lib().w4a16_quantize_pack_mode(
        _dev_ptr(W, "W", torch.float16), _dev_ptr(s, "s", torch.float16, K), N, K, mode,
        _dev_ptr(out.wq, "wq", torch.uint8, wq_b),
        _dev_ptr(out.scales, "scales", torch.float16, sc_b // 2),
        _dev_ptr(out.zeros, "zeros", torch.float16, z_b // 2), _stream_handle(W.device))
    if rc:
        raise W4A16Error(rc, "w4a16_quantize_pack")
    out.wbits = 8 if mode == QUANT_ASYM8 else 4
    return out


def page_outlier_count(N: int, K: int) -> int:
    """The 0.1% share of an N x K matrix kept in fp16 by the mhpq.cn notes (sec.2.2),
    rounded to the nearest integer."""
    return (N * K + 500) // 1000


def w4a16_outlier_workspace_size(N: int, K: int) -> int:
    n = ctypes.c_size_t()
    rc = lib().w4a16_outlier_workspace_size(N, K, ctypes.byref(n))
    if rc:
        raise W4A16Error(rc, "w4a16_outlier_workspace_size")
    return n.value


def w4a16_quantize_pack_outliers(W, s=None, count: int | None = None,
                                 mode: int = QUANT_ASYM) -> PackedWeight:
    """Keep the `count` largest |W / s| of fp16 W[N][K] in fp16 (default: the 0.1% share)
    and quantize the rest into a PackedWeight that carries the outliers."""
    torch = _torch()
    if W.dim() != 2:
        raise ValueError("W must be 2-D [N][K]")
    N, K = W.shape
    if count is None:
        count = page_outlier_count(N, K)
    wq_b, sc_b, z_b = w4a16_packed_sizes(N, K, mode)
    dev = W.device
    pw = PackedWeight(torch.empty(wq_b, dtype=torch.uint8, device=dev),
                      torch.empty(sc_b // 2, dtype=torch.float16, device=dev),
                      torch.empty(z_b // 2, dtype=torch.float16, device=dev), N, K,
                      torch.empty(N + 1, dtype=torch.int32, device=dev),
                      torch.empty(max(count, 1), dtype=torch.int32, device=dev)[:count],
                      torch.empty(max(count, 1), dtype=torch.float16, device=dev)[:count],
                      8 if mode == QUANT_ASYM8 else 4)
    ws = torch.empty(w4a16_outlier_workspace_size(N, K), dtype=torch.uint8, device=dev)
    rc = lib().w4a16_quantize_pack_outliers(
        _dev_ptr(W, "W", torch.float16), _dev_ptr(s, "s", torch.float16, K), N, K, mode, count,
        _dev_ptr(pw.wq, "wq", torch.uint8, wq_b),
        _dev_ptr(pw.scales, "scales", torch.float16, sc_b // 2),
        _dev_ptr(pw.zeros, "zeros", torch.float16, z_b // 2),
        _dev_ptr(pw.o_row_ptr, "o_row_ptr", torch.int32, N + 1),
        ctypes.c_void_p(pw.o_col.data_ptr()), ctypes.c_void_p(pw.o_val.data_ptr()),
        _dev_ptr(ws, "workspace", torch.uint8), ws.numel(), _stream_handle(dev))
    if rc:
        raise W4A16Error(rc, "w4a16_quantize_pack_outliers")
    return pw


def w4a16_quantize_pack_gptq(W, s, Xcal, damp: float = 0.01) -> PackedWeight:
    """GPTQ quantize-and-pack of fp16 W[N][K] (AWQ s[K] or None) with fp16 calibration
    activations Xcal[n][K]: the packed format of w4a16_quantize_pack."""
    torch = _torch()
    if W.dim() != 2 or Xcal.dim() != 2 or Xcal.shape[1] != W.shape[1]:
        raise ValueError("W must be [N][K] and Xcal [n][K]")
    N, K = W.shape
    n = Xcal.shape[0]
    wq_b, sc_b, z_b = w4a16_packed_sizes(N, K)
    dev = W.device
    pw = PackedWeight(torch.empty(wq_b, dtype=torch.uint8, device=dev),
                      torch.empty(sc_b // 2, dtype=torch.float16, device=dev),
                      torch.empty(z_b // 2, dtype=torch.float16, device=dev), N, K)
    nb = ctypes.c_size_t()
    rc = lib().w4a16_gptq_workspace_size(N, K, n, ctypes.byref(nb))
    if rc:
        raise W4A16Error(rc, "w4a16_gptq_workspace_size")
    ws = torch.empty(nb.value, dtype=torch.uint8, device=dev)
    rc = lib().w4a16_quantize_pack_gptq(
        _dev_ptr(W, "W", torch.float16), _dev_ptr(s, "s", torch.float16, K), N, K,
        _dev_ptr(Xcal, "Xcal", torch.float16), n, float(damp),
        _dev_ptr(pw.wq, "wq", torch.uint8, wq_b),
        _dev_ptr(pw.scales, "scales", torch.float16, sc_b // 2),
        _dev_ptr(pw.zeros, "zeros", torch.float16, z_b // 2),
        _dev_ptr(ws, "workspace", torch.uint8), ws.numel(), _stream_handle(dev))
    if rc:
        raise W4A16Error(rc, "w4a16_quantize_pack_gptq")
    return pw


def w4a16_gemm_path(X, pw: PackedWeight, s=None, path: int = PATH_AUTO, out=None):
    """Y[M][N] = X[M][K] . dequant(pw)^T (fp16), on the current stream, asynchronously.
    (Without fp16 outliers: the forced-path entry point does not take them.)"""
    torch = _torch()
    if pw.outlier_ptrs()[0] is not None:
        raise ValueError("w4a16_gemm_path takes no fp16 outliers; use w4a16_gemm")
    if pw.wbits != 4:
        raise ValueError("w4a16_gemm_path takes INT4 codes only; use w4a16_gemm")
    if X.dim() != 2 or X.shape[1] != pw.K:
        raise ValueError("X must be [M][K] with K matching the packed weight")
    M = X.shape[0]
    if out is None:
        out = torch.empty((M, pw.N), dtype=torch.float16, device=X.device)
    elif tuple(out.shape) != (M, pw.N):
        raise ValueError("out must be [M][N]")
    rc = lib().w4a16_gemm_path(
        _dev_ptr(X, "X", torch.float16), _dev_ptr(pw.wq, "wq", torch.uint8),
        _dev_ptr(pw.scales, "scales", torch.float16), _dev_ptr(pw.zeros, "zeros", torch.float16),
        _dev_ptr(s, "s", torch.float16, pw.K), _dev_ptr(out, "out", torch.float16),
        M, pw.N, pw.K, path, _stream_handle(X.device))
    if rc:
        raise W4A16Error(rc, "w4a16_gemm")
    return out


def w4a16_gemm(X, pw: PackedWeight, s=None, out=None):
    """Y[M][N] = X[M][K] . dequant(pw)^T through the grouped entry point with a workspace,
    so large-M calls may split K across workgroups.  X (and Y) fp16 or bf16."""
    torch = _torch()
    if X.dim() != 2 or X.shape[1] != pw.K:
        raise ValueError("X must be [M][K] with K matching the packed weight")
    if out is None:
        out = torch.empty((X.shape[0], pw.N), dtype=X.dtype, device=X.device)
    GroupedCall([(X, pw, s, out)])()
    return out


class GroupedCall:
    """A prepared w4a16_gemm_grouped_ws call: the problem array is marshalled and the
    workspace (w4a16_gemm_workspace_size bytes, a torch tensor owned by this object)
    allocated once, so each call is a single C call on the current stream (for
    captured or repeated launches over the same buffers).  Items are (X,
    PackedWeight, s or None, Y).  Calls of one object must not overlap in time on
    different streams, since they share the workspace.  With ``static=True`` the call
    goes to w4a16_gemm_grouped_static instead: no workspace is allocated here, the
    library's own static scratch serves (all such calls on a GPU share it).  With
    ``workspace=False`` it goes to w4a16_gemm_grouped, which takes no workspace
    argument (the library's event-ordered shared scratch serves when it fits).  A
    uint8 device tensor as ``workspace`` is used instead of a new one (calls that
    share it must not overlap in time)."""

    def __init__(self, items, stream=None, workspace=True, static=False):
        torch = _torch()
        self.items = list(items)  # keep the tensors alive
        # a fixed HIP stream (e.g. torch.cuda.current_stream().cuda_stream) saves
        # looking up torch's current stream on every call
        self.stream = None if stream is None else ctypes.c_void_p(stream)
        self.array = (Problem * len(self.items))()
        for i, (X, pw, s, Y) in enumerate(self.items):
            if X.dim() != 2 or X.shape[1] != pw.K or tuple(Y.shape) != (X.shape[0], pw.N):
                raise ValueError(f"problem {i}: X must be [M][K] and Y [M][N]")
            if X.dtype not in (torch.float16, torch.bfloat16):
                raise TypeError(f"problem {i}: X must be float16 or bfloat16")
            self.array[i] = Problem(
                _dev_ptr(X, "X", X.dtype),
                _dev_ptr(pw.wq, "wq", torch.uint8, pw.N * pw.K * pw.wbits // 8),
                _dev_ptr(pw.scales, "scales", torch.float16),
                _dev_ptr(pw.zeros, "zeros", torch.float16), _dev_ptr(s, "s", torch.float16, pw.K),
                _dev_ptr(Y, "Y", X.dtype), X.shape[0], pw.N, pw.K, *pw.outlier_ptrs(),
                DTYPE_BF16 if X.dtype == torch.bfloat16 else DTYPE_F16, pw.wbits)
        self.device = self.items[0][0].device if self.items else None
        self.ws, self.ws_ptr, self.ws_bytes = None, None, 0
        self.static = static
        self.use_ws = workspace is not False
        if self.use_ws and self.items and not static:
            nb = ctypes.c_size_t()
            rc = lib().w4a16_gemm_workspace_size(self.array, len(self.items), ctypes.byref(nb))
            if rc:
                raise W4A16Error(rc, "w4a16_gemm_workspace_size")
            if nb.value:
                if isinstance(workspace, torch.Tensor):  # a caller's buffer, shared by calls
                    if (not workspace.is_cuda or workspace.dtype != torch.uint8
                            or not workspace.is_contiguous() or workspace.numel() < nb.value):
                        raise ValueError(f"workspace must be a contiguous uint8 device tensor "
                                         f"of at least {nb.value} bytes")
                    self.ws = workspace
                else:
                    self.ws = torch.empty(nb.value, dtype=torch.uint8, device=self.device)
                self.ws_ptr, self.ws_bytes = self.ws.data_ptr(), nb.value

    def __call__(self):
        if not self.items:
            return
        st = self.stream if self.stream is not None else _stream_handle(self.device)
        if self.static:
            rc = lib().w4a16_gemm_grouped_static(self.array, len(self.items), st)
            if rc:
                raise W4A16Error(rc, "w4a16_gemm_grouped_static")
            return
        if not self.use_ws:
            rc = lib().w4a16_gemm_grouped(self.array, len(self.items), st)
            if rc:
                raise W4A16Error(rc, "w4a16_gemm_grouped")
            return
        rc = lib().w4a16_gemm_grouped_ws(self.array, len(self.items), self.ws_ptr,
                                         self.ws_bytes, st)
        if rc:
            raise W4A16Error(rc, "w4a16_gemm_grouped_ws")


def w4a16_gemm_grouped(items):
    """Several independent Y = X . dequant(pw)^T in as few launches as possible.
    items: list of (X, PackedWeight, s or None); returns the list of Y tensors."""
    torch = _torch()
    full = [(X, pw, s, torch.empty((X.shape[0], pw.N), dtype=X.dtype, device=X.device))
            for (X, pw, s) in items]
    GroupedCall(full)()
    return [it[3] for it in full]


def w4a16_gemm_grouped_static(items):
    """w4a16_gemm_grouped with the library's static scratch as the workspace (no device
    allocation by the library; outputs are allocated here).  items: list of (X,
    PackedWeight, s or None); returns the list of Y tensors."""
    torch = _torch()
    full = [(X, pw, s, torch.empty((X.shape[0], pw.N), dtype=X.dtype, device=X.device))
            for (X, pw, s) in items]
    GroupedCall(full, static=True)()
    return [it[3] for it in full]


def w4a16_spec_verify_workspace_size(B: int, K: int, V: int) -> int:
    n = ctypes.c_size_t()
    rc = lib().w4a16_spec_verify_workspace_size(B, K, V, ctypes.byref(n))
    if rc:
        raise W4A16Error(rc, "w4a16_spec_verify_workspace_size")
    return n.value


class SpecVerifyCall:
    """A prepared w4a16_spec_verify call over fixed buffers: shapes are checked, pointers
    marshalled and the workspace allocated once, so each call is a single C call (two
    kernel launches) on the stream.

    p_target fp32 [B][K+1][V], p_draft fp32 [B][K][V], draft int32 [B][K], u_accept fp32
    [B][K], u_sample fp32 [B] (device tensors).  Each call writes n_accepted and token,
    int32 [B] each: the number of accepted drafts and the token drawn after them (-1 if
    the row it is drawn from has no mass).  `workspace` (uint8 device tensor of at least
    w4a16_spec_verify_workspace_size bytes) is allocated when not given; calls sharing a
    workspace must not overlap in time on different streams."""

    def __init__(self, p_target, p_draft, draft, u_accept, u_sample, out=None, workspace=None,
                 stream=None):
        torch = _torch()
        if p_target.dim() != 3:
            raise ValueError("p_target must be [B][K+1][V]")
        B, K1, V = p_target.shape
        K = K1 - 1
        if K < 0:
            raise ValueError("p_target needs at least one position")
        if tuple(p_draft.shape) != (B, K, V) or tuple(draft.shape) != (B, K) \
                or tuple(u_accept.shape) != (B, K) or tuple(u_sample.shape) != (B,):
            raise ValueError("p_draft [B][K][V], draft [B][K], u_accept [B][K], u_sample [B]")
        ws_bytes = w4a16_spec_verify_workspace_size(B, K, V)
        dev = p_target.device
        if workspace is None:
            workspace = torch.empty(max(ws_bytes, 1), dtype=torch.uint8, device=dev)
        elif workspace.numel() < ws_bytes:
            raise ValueError(f"workspace needs {ws_bytes} bytes")
        if out is None:
            out = (torch.empty(B, dtype=torch.int32, device=dev),
                   torch.empty(B, dtype=torch.int32, device=dev))
        self.out = out
        self.keep = (p_target, p_draft, draft, u_accept, u_sample, workspace)
        self.device = dev
        self.stream = None if stream is None else ctypes.c_void_p(stream)
        self.args = (
            _dev_ptr(p_target, "p_target", torch.float32),
            _dev_ptr(p_draft, "p_draft", torch.float32),
            _dev_ptr(draft, "draft", torch.int32), _dev_ptr(u_accept, "u_accept", torch.float32),
            _dev_ptr(u_sample, "u_sample", torch.float32), B, K, V,
            _dev_ptr(workspace, "workspace", torch.uint8), workspace.numel(),
            _dev_ptr(out[0], "n_accepted", torch.int32, B),
            _dev_ptr(out[1], "token", torch.int32, B))

    def __call__(self):
        st = self.stream if self.stream is not None else _stream_handle(self.device)
        rc = lib().w4a16_spec_verify(*self.args, st)
        if rc:
            raise W4A16Error(rc, "w4a16_spec_verify")
        return self.out


def w4a16_spec_verify(p_target, p_draft, draft, u_accept, u_sample, out=None, workspace=None):
    """Speculative-sampling verification of B sequences on the current stream; returns
    (n_accepted, token).  Arguments as for SpecVerifyCall."""
    return SpecVerifyCall(p_target, p_draft, draft, u_accept, u_sample, out, workspace)()


# ---- fused linear layers and their backward passes -------------------------------------

def _refuse_grad(t, name):
    """These calls record no graph: a tensor whose gradient autograd expects would lose it
    without a word.  (An autograd.Function's forward and backward run without grad mode.)"""
    if t.requires_grad and _torch().is_grad_enabled():
        raise ValueError(f"{name} requires grad, and the fused calls record no graph: call them "
                         "from an autograd.Function (forward here, backward through the "
                         "*_backward calls) or under torch.no_grad()")


def _act_dtype(t, name):
    """The activations' type of tensor t: torch.float16 or torch.bfloat16."""
    torch = _torch()
    if not isinstance(t, torch.Tensor) or t.dtype not in (torch.float16, torch.bfloat16):
        raise TypeError(f"{name} must be a float16 or bfloat16 tensor")
    _refuse_grad(t, name)
    return t.dtype


def _dtype_code(dtype):
    return DTYPE_BF16 if dtype == _torch().bfloat16 else DTYPE_F16


def _shaped_ptr(t, name, dtype, shape, device):
    """Device pointer of an optional tensor of this type, shape and device."""
    if t is None:
        return None
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    p = _dev_ptr(t, name, dtype)
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    _refuse_grad(t, name)
    return p


def _problem(X, pw, s, y_ptr, device):
    torch = _torch()
    if X.dim() != 2 or X.shape[1] != pw.K:
        raise ValueError("X must be [M][K] with K matching the packed weight")
    meta = (pw.N * (-(-(pw.K // GROUP) // 4) * 4),)
    return Problem(
        _dev_ptr(X, "X", X.dtype),
        _shaped_ptr(pw.wq, "wq", torch.uint8, (pw.N * pw.K * pw.wbits // 8,), device),
        _shaped_ptr(pw.scales, "scales", torch.float16, meta, device),
        _shaped_ptr(pw.zeros, "zeros", torch.float16, meta, device),
        _shaped_ptr(s, "s", torch.float16, (pw.K,), device), y_ptr, X.shape[0], pw.N, pw.K,
        *pw.outlier_ptrs(), _dtype_code(X.dtype), pw.wbits)


class _PreparedCall:
    """One C call over fixed buffers on one device, with a workspace of its own (or a
    caller's uint8 device tensor).  Calls that share a workspace must not overlap in time,
    nor may replays of captured calls that share one."""

    def _prepare(self, device, nbytes, workspace, stream):
        torch = _torch()
        self.device = device
        self.stream = None if stream is None else ctypes.c_void_p(stream)
        self.ws, self.ws_ptr, self.ws_bytes = None, None, 0
        if nbytes == 0:
            return
        if workspace is None:
            workspace = torch.empty(nbytes, dtype=torch.uint8, device=device)
        elif (not workspace.is_cuda or workspace.dtype != torch.uint8 or workspace.device != device
              or not workspace.is_contiguous() or workspace.numel() < nbytes):
            raise ValueError(f"workspace must be a contiguous uint8 tensor of at least {nbytes} "
                             f"bytes on {device}")
        self.ws, self.ws_ptr, self.ws_bytes = workspace, workspace.data_ptr(), nbytes

    def _bind(self, name, *args):
        """The C function and its arguments up to the stream: what is left for each call
        is the current stream and device."""
        self.name, self.function = name, getattr(lib(), name)
        self.args = (*args, self.ws_ptr, self.ws_bytes)
        self.index = None if self.device is None else self.device.index
        cuda = _torch()._C  # the raw lookups, without a Stream object (1.5 us less per call)
        self.current_stream = getattr(cuda, "_cuda_getCurrentRawStream", None)
        self.current_device = getattr(cuda, "_cuda_getDevice", _torch().cuda.current_device)

    def __call__(self):
        if self.stream is not None:
            st = self.stream
        elif self.current_stream is not None:
            st = self.current_stream(self.index)
        else:
            st = _stream_handle(self.device)
        if self.current_device() == self.index:
            rc = self.function(*self.args, st)
        else:
            with _torch().cuda.device(self.device):
                rc = self.function(*self.args, st)
        if rc:
            raise W4A16Error(rc, self.name)

    @staticmethod
    def _size(name, *args):
        n = ctypes.c_size_t()
        rc = getattr(lib(), name)(*args, ctypes.byref(n))
        if rc:
            raise W4A16Error(rc, name)
        return n.value


@dataclass
class Epilogue:
    """What a linear layer does to its product Z = X . dequant(pw)^T + bias before it is
    stored: Y = residual + act(Z).  bias [N], residual [M][N] (may be Y itself) and preact
    [M][N] (receives Z) are of X's type; act is one of the ACT_* constants."""
    bias: "object" = None
    act: int = ACT_NONE
    residual: "object" = None
    preact: "object" = None


class LinearCall(_PreparedCall):
    """A prepared w4a16_linear call.  Items are (X, PackedWeight, s or None, Y, Epilogue);
    problems of one call share launches as in GroupedCall.  All tensors are on one device;
    each call runs on the current stream, or on ``stream`` (a HIP stream handle)."""

    def __init__(self, items, stream=None, workspace=None):
        self.items = list(items)  # keep the tensors alive
        n = len(self.items)
        self.problems, self.epilogues = (Problem * n)(), (EpilogueStruct * n)()
        device = self.items[0][0].device if n else None
        for i, (X, pw, s, Y, e) in enumerate(self.items):
            dt = _act_dtype(X, f"problem {i}: X")
            shape = (X.shape[0], pw.N)
            if X.device != device:
                raise ValueError(f"problem {i}: X must be on {device}")
            self.problems[i] = _problem(X, pw, s, _shaped_ptr(Y, "Y", dt, shape, device), device)
            self.epilogues[i] = EpilogueStruct(
                _shaped_ptr(e.bias, "bias", dt, (pw.N,), device),
                _shaped_ptr(e.residual, "residual", dt, shape, device),
                _shaped_ptr(e.preact, "preact", dt, shape, device), e.act)
        nbytes = self._size("w4a16_linear_workspace_size", self.problems, self.epilogues, n)
        self._prepare(device, nbytes, workspace, stream)
        self._bind("w4a16_linear", self.problems, self.epilogues, n)

    def __call__(self):
        if self.items:
            super().__call__()


def w4a16_linear(X, pw: PackedWeight, s=None, bias=None, act=ACT_NONE, residual=None, out=None,
                 preact=None):
    """Y = residual + act(X . dequant(pw)^T + bias) on the current stream; X fp16 or bf16
    [M][K].  preact, when given, receives the pre-activation for a backward pass.  Like all
    fused calls it is not differentiable by itself: in grad mode a tensor that requires grad
    is refused (w4a16_linear_backward gives the gradients)."""
    if out is None:
        out = _torch().empty((X.shape[0], pw.N), dtype=X.dtype, device=X.device)
    LinearCall([(X, pw, s, out, Epilogue(bias, act, residual, preact))])()
    return out


class GatedCall(_PreparedCall):
    """A prepared w4a16_gated call: H = act(G) * U with G = X . dequant(gate)^T + bias_gate
    and U = X . dequant(up)^T + bias_up, both products in one pass over X.  preact: a pair
    of [M][N] tensors that receive G and U, or None."""

    def __init__(self, X, gate, up, s, H, act=ACT_SILU, bias_gate=None, bias_up=None, preact=None,
                 stream=None, workspace=None):
        dt, device = _act_dtype(X, "X"), X.device
        if (gate.N, gate.K, gate.wbits) != (up.N, up.K, up.wbits):
            raise ValueError("gate and up must have the same shape and code width")
        shape = (X.shape[0], gate.N)
        G, U = preact if preact is not None else (None, None)
        self.keep = (X, gate, up, s, H, bias_gate, bias_up, G, U)
        self.gate = _problem(X, gate, s, _shaped_ptr(G, "preact[0]", dt, shape, device), device)
        self.up = _problem(X, up, s, _shaped_ptr(U, "preact[1]", dt, shape, device), device)
        args = (ctypes.byref(self.gate), ctypes.byref(self.up),
                _shaped_ptr(bias_gate, "bias_gate", dt, (gate.N,), device),
                _shaped_ptr(bias_up, "bias_up", dt, (gate.N,), device), act,
                _shaped_ptr(H, "H", dt, shape, device))
        nbytes = self._size("w4a16_gated_workspace_size", *args[:2])
        self._prepare(device, nbytes, workspace, stream)
        self._bind("w4a16_gated", *args)


def w4a16_gated(X, gate: PackedWeight, up: PackedWeight, s=None, act=ACT_SILU, bias_gate=None,
                bias_up=None, out=None, preact=None):
    """H = act(X . dequant(gate)^T + bias_gate) * (X . dequant(up)^T + bias_up) on the
    current stream.  preact: a pair of tensors that receive the two pre-activations."""
    if out is None:
        out = _torch().empty((X.shape[0], gate.N), dtype=X.dtype, device=X.device)
    GatedCall(X, gate, up, s, out, act, bias_gate, bias_up, preact)()
    return out


@dataclass
class TransposedWeight:
    """Transposed copy of a PackedWeight for the backward passes (layout: w4a16_transpose in
    include/w4a16.h)."""
    wt: "object"
    meta: "object"
    N: int
    K: int
    wbits: int = 4


def w4a16_transpose(pw: PackedWeight) -> TransposedWeight:
    """The transposed copy that the backward passes read, made once per weight (on the
    current stream).  Weights with fp16 outliers have none."""
    torch = _torch()
    if pw.outlier_ptrs()[0] is not None:
        raise ValueError("weights with fp16 outliers have no transposed form")
    a, b = ctypes.c_size_t(), ctypes.c_size_t()
    rc = lib().w4a16_transposed_sizes(pw.N, pw.K, pw.wbits, ctypes.byref(a), ctypes.byref(b))
    if rc:
        raise W4A16Error(rc, "w4a16_transposed_sizes")
    dev = pw.wq.device
    meta = (pw.N * (-(-(pw.K // GROUP) // 4) * 4),)
    src = (_shaped_ptr(pw.wq, "wq", torch.uint8, (pw.N * pw.K * pw.wbits // 8,), dev),
           _shaped_ptr(pw.scales, "scales", torch.float16, meta, dev),
           _shaped_ptr(pw.zeros, "zeros", torch.float16, meta, dev))
    out = TransposedWeight(torch.empty(a.value, dtype=torch.uint8, device=dev),
                           torch.empty(b.value, dtype=torch.uint8, device=dev), pw.N, pw.K,
                           pw.wbits)
    with torch.cuda.device(dev):
        rc = lib().w4a16_transpose(*src, pw.N, pw.K, pw.wbits, _dev_ptr(out.wt, "wt"),
                                   _dev_ptr(out.meta, "meta"), _stream_handle(dev))
    if rc:
        raise W4A16Error(rc, "w4a16_transpose")
    return out


@dataclass
class BackwardTerm:
    """One layer of a backward call: dZ = dY * act'(preact), dbias = column sums of dZ.
    With ACT_NONE dZ is dY itself, and preact and dZ must be None.  dbias: fp32 [N] output
    or None."""
    dY: "object"
    wt: TransposedWeight
    act: int = ACT_NONE
    preact: "object" = None
    dZ: "object" = None
    dbias: "object" = None

    def struct(self, dt, shape, device):
        torch = _torch()
        w = self.wt
        ng = -(-w.N // GROUP)
        return BackwardTermStruct(
            _shaped_ptr(self.dY, "dY", dt, shape, device),
            _shaped_ptr(self.preact, "preact", dt, shape, device),
            _shaped_ptr(self.dZ, "dZ", dt, shape, device),
            _shaped_ptr(self.dbias, "dbias", torch.float32, (w.N,), device),
            _shaped_ptr(w.wt, "wt", torch.uint8, (ng * GROUP * w.K * w.wbits // 8,), device),
            _shaped_ptr(w.meta, "meta", torch.uint8, (ng * (w.K // GROUP) * 512,), device),
            w.N, self.act, w.wbits)


class LinearBackwardCall(_PreparedCall):
    """A prepared w4a16_linear_backward call: dX = add + s * sum over the terms of dZ . D,
    and each term's dZ and dbias.  The terms (1 to 4 BackwardTerm) are the layers that read
    the same X with the same s.  dX None: only dZ and dbias; add may be dX itself, and a dZ
    its own term's dY or preact (where neither add nor another term is in that buffer)."""

    def __init__(self, terms, s, dX, add=None, stream=None, workspace=None):
        torch = _torch()
        self.keep = (list(terms), s, dX, add)
        terms = self.keep[0]
        if not terms:
            raise ValueError("at least one term")
        dt, device = _act_dtype(terms[0].dY, "dY"), terms[0].dY.device
        M, K = terms[0].dY.shape[0], terms[0].wt.K
        if any(t.wt.K != K for t in terms):
            raise ValueError("the terms' weights must have the same K")
        self.terms = (BackwardTermStruct * len(terms))()
        for i, t in enumerate(terms):
            self.terms[i] = t.struct(dt, (M, t.wt.N), device)
        args = (self.terms, len(terms), _shaped_ptr(s, "s", torch.float16, (K,), device),
                _shaped_ptr(add, "add", dt, (M, K), device),
                _shaped_ptr(dX, "dX", dt, (M, K), device), M, K, _dtype_code(dt))
        nbytes = self._size("w4a16_linear_backward_workspace_size", self.terms, len(terms), M, K,
                            _dtype_code(dt))
        self._prepare(device, nbytes, workspace, stream)
        self._bind("w4a16_linear_backward", *args)


def w4a16_linear_backward(dY, wt: TransposedWeight, s=None, act=ACT_NONE, preact=None, add=None,
                          bias_grad=False):
    """Backward of w4a16_linear on the current stream: (dX, dZ, dbias).  dZ is dY itself for
    ACT_NONE; dbias (fp32) is None unless bias_grad.  The residual's gradient is dY."""
    torch = _torch()
    M = dY.shape[0]
    dX = torch.empty((M, wt.K), dtype=dY.dtype, device=dY.device)
    dZ = torch.empty_like(dY) if act != ACT_NONE else None
    db = torch.empty(wt.N, dtype=torch.float32, device=dY.device) if bias_grad else None
    LinearBackwardCall([BackwardTerm(dY, wt, act, preact, dZ, db)], s, dX, add)()
    return dX, dY if dZ is None else dZ, db


class GatedBackwardCall(_PreparedCall):
    """A prepared w4a16_gated_backward call: dG = dH * U * act'(G), dU = dH * act(G),
    dX = add + s * (dG . Dg + dU . Du), and the fp32 column sums of dG and dU.  dG may be G
    and dU may be U, or one of them dH (where add is not dH); dX None: only dG, dU and the
    sums."""

    def __init__(self, dH, G, U, gate: TransposedWeight, up: TransposedWeight, s, dX, dG, dU,
                 act=ACT_SILU, add=None, dbias_gate=None, dbias_up=None, stream=None,
                 workspace=None):
        torch = _torch()
        dt, device = _act_dtype(dH, "dH"), dH.device
        if (gate.N, gate.K, gate.wbits) != (up.N, up.K, up.wbits):
            raise ValueError("gate and up must have the same shape and code width")
        M, K = dH.shape[0], gate.K
        shape = (M, gate.N)
        self.keep = (dH, G, U, gate, up, s, dX, dG, dU, add, dbias_gate, dbias_up)
        self.gate = BackwardTerm(None, gate, act, G, dG, dbias_gate).struct(dt, shape, device)
        self.up = BackwardTerm(None, up, ACT_NONE, U, dU, dbias_up).struct(dt, shape, device)
        refs = (ctypes.byref(self.gate), ctypes.byref(self.up))
        args = (_shaped_ptr(dH, "dH", dt, shape, device), *refs,
                _shaped_ptr(s, "s", torch.float16, (K,), device),
                _shaped_ptr(add, "add", dt, (M, K), device),
                _shaped_ptr(dX, "dX", dt, (M, K), device), M, K, _dtype_code(dt))
        nbytes = self._size("w4a16_gated_backward_workspace_size", *refs, M, K, _dtype_code(dt))
        self._prepare(device, nbytes, workspace, stream)
        self._bind("w4a16_gated_backward", *args)


def w4a16_gated_backward(dH, G, U, gate: TransposedWeight, up: TransposedWeight, s=None,
                         act=ACT_SILU, add=None, bias_grad=False):
    """Backward of w4a16_gated on the current stream, from dH and the saved pre-activations:
    (dX, dG, dU, dbias_gate, dbias_up); the bias gradients (fp32) are None unless bias_grad."""
    torch = _torch()
    dX = torch.empty((dH.shape[0], gate.K), dtype=dH.dtype, device=dH.device)
    dG, dU = torch.empty_like(dH), torch.empty_like(dH)
    db = [torch.empty(gate.N, dtype=torch.float32, device=dH.device) if bias_grad else None
          for _ in range(2)]
    GatedBackwardCall(dH, G, U, gate, up, s, dX, dG, dU, act, add, *db)()
    return dX, dG, dU, db[0], db[1]


from . import experts  # noqa: E402  (it takes the pieces above)
from .experts import *  # noqa: E402,F401,F403

__all__ += experts.__all__
