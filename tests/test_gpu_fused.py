"""Fused linear layers and their backward passes on the GPU against the fp64 oracle.

Tolerances.  u is the activations' unit roundoff (2^-11 fp16, 2^-8 bf16).  A product
rounds X * s, the dequantized weight (tiled and backward kernels) and the output once
each, u relative to each, and sums in fp32; its relative L2 error is held to the bounds of
the plain products (REL_L2 of gpu_helpers: three independent roundings and margin).
  * element by element: |Z' - Z| <= (2 u + 2 u^2 + (K + 8) 2^-24) * A, with
    A = |X s| |q - z| scale summed in fp64, before the output's own rounding of u |Z'|,
    plus 2^-25 (half the smallest fp16) per output.
  * act: the slopes of every activation lie in [-0.2, 1.2], its fp32 evaluation is within
    2^-19 * (1 + |z|); so Y moves by at most 1.2 e_Z, and H = act(G) U by
    1.2 e_G (|U| + e_U) + |act(G)| e_U.  Relative L2: with G and U of unit size the ratio
    of rms(act') |U| to rms(act(G) U) is at most 1.2 / 0.34 < 4 (silu at rms 1 is 0.34 or
    more of its input), so H and Y are held to 5 x REL_L2.
  * dZ: u |dZ| + 2^-18 |dY| (1 + |z|) (1 + |u|) + 2^-25.
  * dX: the products' bound with dZ in the place of X s (rounded once), applied to the
    oracle's unrounded dZ, times s, plus u |dX|.
  * bias sums: fp32, at most M terms: (M + 8) 2^-24 * sum |dZ| + the fp32 evaluation above.
"""
import ctypes

import numpy as np
import pytest

import oracle
import weight_only_int4_group_amd as w4
from oracle import fused as of
from oracle import outliers as ol
from tests.gpu_helpers import (MAX_REL_BF16, REL_L2, REL_L2_BF16, errors, note, to_dev, to_host,
                               torch_cuda)
from workloads import (activations, activations_bf16, awq_scales, bf16_bits_to_f64, to_bf16_bits,
                       weights)

pytestmark = pytest.mark.gpu

U = {"fp16": 2.0 ** -11, "bf16": 2.0 ** -8}
REL = {"fp16": REL_L2, "bf16": REL_L2_BF16}
TINY = 2.0 ** -25
ACT = {n: getattr(w4, "ACT_" + n.upper()) for n in of.ACTS}
_PACKED = {}


class Weight:
    """A packed weight on the GPU and its fp64 value."""

    def __init__(self, key, N, K, awq, bits=4, count=0):
        torch_cuda()
        W, s = weights(41, key, N, K), awq_scales(41, key % 2, K) if awq else None
        self.s = s
        self.sd = None if s is None else to_dev(s)
        mode = w4.QUANT_ASYM8 if bits == 8 else w4.QUANT_ASYM
        if count:
            self.pw = w4.w4a16_quantize_pack_outliers(to_dev(W), self.sd, count, mode)
        else:
            self.pw = w4.w4a16_quantize_pack(to_dev(W), self.sd, mode=mode)
        self.q = (oracle.unpack_codes8 if bits == 8 else oracle.unpack_codes)(to_host(self.pw.wq), N, K)
        self.scales = oracle.unpack_meta(to_host(self.pw.scales), N, K)
        self.zeros = oracle.unpack_meta(to_host(self.pw.zeros), N, K)
        self.D = oracle.dequantize(self.q, self.scales, self.zeros)
        self.W = self.D if s is None else self.D * s.astype(np.float64)
        if count:
            rp, col = to_host(self.pw.o_row_ptr), to_host(self.pw.o_col)
            rows = np.repeat(np.arange(N), np.diff(rp))
            self.W = self.W.copy()
            self.W[rows, col] = to_host(self.pw.o_val).astype(np.float64)


def weight(key, N, K, awq=False, bits=4, count=0):
    k = (key, N, K, awq, bits, count)
    if k not in _PACKED:
        if len(_PACKED) > 24:
            _PACKED.clear()
        _PACKED[k] = Weight(*k)
    return _PACKED[k]


def act_array(dtype, key, M, N, scale=1.0):
    """(device tensor, fp64 values) of M x N normal values of the activations' type."""
    torch = torch_cuda()
    x = np.random.default_rng([43, key, M, N]).standard_normal((M, N)).astype(np.float32) * np.float32(scale)
    if dtype == "fp16":
        h = x.astype(np.float16)
        return to_dev(h), h.astype(np.float64)
    b = to_bf16_bits(x)
    return to_dev(b.view(np.int16)).view(torch.bfloat16), bf16_bits_to_f64(b)


def values(t):
    torch = torch_cuda()
    torch.cuda.synchronize()
    return t.double().cpu().numpy()


def guarded(dtype, M, N):
    """An [M][N] output at the start of a buffer whose rows behind it hold a sentinel."""
    torch = torch_cuda()
    dt = torch.float16 if dtype == "fp16" else torch.bfloat16
    buf = torch.full((M + 3, N), 777.0, dtype=dt, device="cuda")
    buf[:M] = float("nan")
    return buf[:M], buf


def check_guard(buf, M):
    assert bool((buf[M:] == 777.0).all()), "rows behind the output were written"


def product_bound(X, W, u, K):
    return (2 * u + 2 * u * u + (K + 8) * 2.0 ** -24) * (np.abs(X) @ np.abs(W).T)


def close(got, ref, bound, tag, rel):
    assert np.isfinite(got).all(), f"{tag}: non-finite"
    bad = np.abs(got - ref) > bound
    assert not bad.any(), f"{tag}: {bad.sum()} of {bad.size} outside, worst " \
        f"{(np.abs(got - ref) / bound).max():.3g} x bound"
    r = errors(got, ref)[0]
    assert r <= rel, f"{tag}: rel-L2 {r:.3e} > {rel:.3e}"


def act_bound(z, e_z):
    return 1.2 * e_z + 2.0 ** -19 * (1 + np.abs(z))


def run_linear(M, N, K, dtype, act="none", bias=False, residual=False, pre=False, awq=False, bits=4,
               count=0, inplace=False, workspace=True):
    torch_cuda()
    note(f"linear M={M} N={N} K={K} {dtype} {act} bias={bias} res={residual} pre={pre} awq={awq} "
         f"bits={bits} outliers={count} inplace={inplace} ws={workspace}")
    w = weight(1, N, K, awq, bits, count)
    X, Xv = act_array(dtype, 1, M, K)
    b, bv = act_array(dtype, 2, 1, N, 0.5)
    b, bv = (b.reshape(N), bv.reshape(N)) if bias else (None, None)
    Y, buf = guarded(dtype, M, N)
    R, Rv = act_array(dtype, 3, M, N) if residual else (None, None)
    if inplace:
        Y.copy_(R)
        R = Y
    Z, zbuf = guarded(dtype, M, N) if pre else (None, None)
    call = w4.LinearCall([(X, w.pw, w.sd, Y, w4.Epilogue(b, ACT[act], R, Z))])
    if not workspace:
        call.args = (*call.args[:-2], None, 0)
    call()
    ref, z = of.linear(Xv, w.W, bv, act, Rv)
    u = U[dtype]
    e = product_bound(Xv, w.W, u, K)
    got = values(Y)
    check_guard(buf, M)
    tag = f"linear {M}x{N}x{K} {dtype}"
    ey = act_bound(z, e) if act != "none" else e
    close(got, ref, ey + u * np.abs(ref) + u * ey + TINY, tag, (5 if act != "none" else 1) * REL[dtype])
    if pre:
        check_guard(zbuf, M)
        close(values(Z), z, e + u * np.abs(z) + u * e + TINY, tag + " Z", REL[dtype])


def run_gated(M, N, K, dtype, act="silu", bias=False, pre=False, awq=False, bits=4, counts=(0, 0),
              workspace=True):
    torch_cuda()
    note(f"gated M={M} N={N} K={K} {dtype} {act} bias={bias} pre={pre} awq={awq} bits={bits} "
         f"outliers={counts} ws={workspace}")
    wg, wu = weight(2, N, K, awq, bits, counts[0]), weight(4, N, K, awq, bits, counts[1])
    X, Xv = act_array(dtype, 1, M, K)
    bg, bgv = act_array(dtype, 5, 1, N, 0.5)
    bu, buv = act_array(dtype, 6, 1, N, 0.5)
    bg, bgv, bu, buv = ((bg.reshape(N), bgv.reshape(N), bu.reshape(N), buv.reshape(N)) if bias
                        else (None,) * 4)
    H, buf = guarded(dtype, M, N)
    saved = [guarded(dtype, M, N) for _ in range(2)] if pre else []
    call = w4.GatedCall(X, wg.pw, wu.pw, wg.sd, H, ACT[act], bg, bu,
                        tuple(t for t, _ in saved) or None)
    if not workspace:
        call.args = (*call.args[:-2], None, 0)
    call()
    ref, g, uu = of.gated(Xv, wg.W, wu.W, act, bgv, buv)
    u = U[dtype]
    eg, eu = product_bound(Xv, wg.W, u, K), product_bound(Xv, wu.W, u, K)
    ea = act_bound(g, eg)
    eh = ea * (np.abs(uu) + eu) + np.abs(of.act(g, act)) * eu
    check_guard(buf, M)
    tag = f"gated {M}x{N}x{K} {dtype}"
    close(values(H), ref, eh + u * np.abs(ref) + u * eh + TINY, tag, 5 * REL[dtype])
    for (t, tb), z, e in zip(saved, (g, uu), (eg, eu)):
        check_guard(tb, M)
        close(values(t), z, e + u * np.abs(z) + u * e + TINY, tag + " saved", REL[dtype])


# shapes: N with a part of a tile column block, K with a part of a metadata quad
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("M", [1, 2, 7, 16, 17, 33, 49, 65, 97, 150])
def test_linear_every_tile_height(M, dtype):
    run_linear(M, 272, 640, dtype, "gelu", bias=True, residual=True, pre=True, awq=M % 2 == 1)


@pytest.mark.parametrize("act", of.ACTS)
@pytest.mark.parametrize("M", [3, 40])
def test_linear_activations(M, act):
    run_linear(M, 48, 384, "fp16", act, bias=True, pre=True)
    run_linear(M, 48, 384, "bf16", act, residual=True)


@pytest.mark.parametrize("M,N,K", [(1, 16, 128), (16, 16, 128), (5, 16, 14336), (9, 48, 14336),
                                   (16, 48, 18944), (1, 2064, 128), (64, 16, 4096), (130, 16, 128)])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_linear_extreme_shapes(M, N, K, dtype):
    run_linear(M, N, K, dtype, "silu", bias=True, residual=True, awq=True)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("M", [1, 9, 40, 200])
def test_linear_int8_codes(M, dtype):
    run_linear(M, 272, 640, dtype, "relu", bias=True, residual=True, pre=True, awq=True, bits=8)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("M,K", [(5, 14464), (16, 4224), (16, 12416)])
def test_streamed_in_ranges_of_k(M, K, dtype, bits):
    """Rows too long for LDS at this M: K in ranges of whole metadata quads (113, 33 and 97
    groups: unequal ranges, a last quad in part), one weight and a gated pair."""
    run_linear(M, 48, K, dtype, "silu", bias=True, residual=True, pre=True, awq=True, bits=bits)
    run_gated(M, 48, K, dtype, "silu", bias=True, pre=True, awq=True, bits=bits)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("M,K", [(5, 14464), (16, 4224)])
def test_streamed_without_room_for_ranges(M, K, dtype, bits):
    """The same rows without a workspace: windows of X * s in one launch."""
    run_linear(M, 48, K, dtype, "silu", bias=True, residual=True, pre=True, awq=True, bits=bits,
               workspace=False)
    run_gated(M, 48, K, dtype, "silu", bias=True, pre=True, awq=True, bits=bits, workspace=False)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("M", [1, 9, 40, 130])
def test_linear_outliers(M, dtype, bits):
    run_linear(M, 272, 640, dtype, "none", bias=True, residual=True, pre=True, awq=True, bits=bits,
               count=900)


@pytest.mark.parametrize("M", [1, 12, 64, 140])
def test_linear_residual_in_place(M):
    run_linear(M, 272, 1152, "bf16", "none", residual=True, inplace=True)
    run_linear(M, 528, 4096, "fp16", "relu", residual=True, inplace=True)


@pytest.mark.parametrize("M", [4, 64, 130])
def test_linear_without_workspace(M):
    run_linear(M, 272, 4096, "fp16", "gelu_tanh", bias=True, residual=True, pre=True, awq=True,
               workspace=False)
    run_linear(M, 272, 4096, "bf16", "gelu_tanh", bias=True, residual=True, pre=True, awq=True,
               workspace=False)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("M", [1, 2, 7, 16, 17, 33, 49, 65, 97, 150])
def test_gated_every_tile_height(M, dtype):
    run_gated(M, 272, 640, dtype, "silu", bias=True, pre=True, awq=M % 2 == 1)


@pytest.mark.parametrize("act", of.ACTS)
@pytest.mark.parametrize("M", [3, 40])
def test_gated_activations(M, act):
    run_gated(M, 48, 384, "fp16", act, bias=True)
    run_gated(M, 48, 384, "bf16", act, pre=True)


@pytest.mark.parametrize("M,N,K", [(1, 16, 128), (16, 16, 128), (5, 16, 14336), (9, 48, 14336),
                                   (16, 48, 18944), (1, 2064, 128), (64, 16, 4096), (130, 16, 128),
                                   (64, 144, 4096)])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_gated_extreme_shapes(M, N, K, dtype):
    run_gated(M, N, K, dtype, "silu", bias=True, awq=True)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("M", [1, 9, 40, 200])
def test_gated_int8_codes(M, dtype):
    run_gated(M, 272, 640, dtype, "gelu", bias=True, pre=True, awq=True, bits=8)


@pytest.mark.parametrize("counts", [(900, 500), (0, 700), (700, 0)])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("M", [1, 9, 40, 130])
def test_gated_outliers(M, dtype, counts):
    run_gated(M, 272, 640, dtype, "silu", bias=True, pre=True, awq=True, counts=counts)
    if counts[0] and counts[1]:
        run_gated(M, 272, 640, dtype, "silu", bits=8, counts=counts)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("M", [130, 200, 256])
def test_blocks_of_128_rows_and_columns(M, dtype, bits):
    """Row counts and widths whose plan is two 128 x 128 blocks on a CU."""
    run_linear(M, 28672, 256, dtype, "silu", bias=True, residual=True, pre=True, awq=True, bits=bits)
    run_gated(M, 14336, 256, dtype, "silu", bias=True, pre=True, awq=True, bits=bits)


@pytest.mark.parametrize("M", [4, 64, 130])
def test_gated_without_workspace(M):
    run_gated(M, 272, 4096, "fp16", "gelu_tanh", bias=True, pre=True, awq=True, workspace=False)
    run_gated(M, 272, 4096, "bf16", "gelu_tanh", bias=True, pre=True, awq=True, workspace=False)


@pytest.mark.parametrize("M,K", [(1, 640), (16, 640), (40, 640), (200, 640), (16, 4224)])
def test_linear_group_of_layers(M, K):
    """q, k and v with biases, and a fourth layer with another epilogue, in one call."""
    torch = torch_cuda()
    dtype = "bf16"
    X, Xv = act_array(dtype, 1, M, K)
    items, refs = [], []
    for i, (N, act) in enumerate([(272, "none"), (48, "none"), (16, "relu"), (144, "silu")]):
        w = weight(10 + i, N, K)
        b, bv = act_array(dtype, 20 + i, 1, N)
        R, Rv = act_array(dtype, 30 + i, M, N) if i == 3 else (None, None)
        Y = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
        items.append((X, w.pw, None, Y, w4.Epilogue(b.reshape(N), ACT[act], R)))
        ref, z = of.linear(Xv, w.W, bv.reshape(N), act, Rv)
        e = act_bound(z, product_bound(Xv, w.W, U[dtype], K))
        refs.append((ref, e + U[dtype] * (np.abs(ref) + e) + TINY))
    note(f"linear group M={M}")
    w4.LinearCall(items)()
    for (X, _, _, Y, _), (ref, bound) in zip(items, refs):
        close(values(Y), ref, bound, f"group M={M}", 5 * REL[dtype])


def run_problems(specs, workspace=True):
    """One w4a16_linear call over (M, N, K, dtype, bits, outliers) problems, each with an
    activation, bias, residual and pre-activation output of its own, each checked."""
    torch = torch_cuda()
    items, checks = [], []
    for i, (M, N, K, dtype, bits, count) in enumerate(specs):
        act, w = of.ACTS[(i + 1) % 5], weight(60 + i, N, K, i % 2 == 0, bits, count)
        X, Xv = act_array(dtype, 100 + i, M, K)
        b, bv = act_array(dtype, 120 + i, 1, N, 0.5)
        R, Rv = act_array(dtype, 140 + i, M, N) if i % 3 != 1 else (None, None)
        (Y, buf), (Z, zbuf) = guarded(dtype, M, N), guarded(dtype, M, N)
        b, bv = (b.reshape(N), bv.reshape(N)) if i % 4 != 2 else (None, None)
        items.append((X, w.pw, w.sd, Y, w4.Epilogue(b, ACT[act], R, Z if i % 2 else None)))
        checks.append((w, Xv, bv, act, Rv, buf, zbuf if i % 2 else None))
    note(f"problems {specs} ws={workspace}")
    call = w4.LinearCall(items)
    if not workspace:
        call.args = (*call.args[:-2], None, 0)
    call()
    for (X, _, _, Y, e), (w, Xv, bv, act, Rv, buf, zbuf), (M, N, K, dtype, bits, count) in zip(
            items, checks, specs):
        u, tag = U[dtype], f"problem {M}x{N}x{K} {dtype} {bits} {count} {act}"
        ref, z = of.linear(Xv, w.W, bv, act, Rv)
        ez = product_bound(Xv, w.W, u, K)
        ey = act_bound(z, ez) if act != "none" else ez
        check_guard(buf, M)
        close(values(Y), ref, ey + u * np.abs(ref) + u * ey + TINY, tag, 5 * REL[dtype])
        if zbuf is not None:
            check_guard(zbuf, M)
            close(values(e.preact), z, ez + u * np.abs(z) + u * ez + TINY, tag + " Z", REL[dtype])


@pytest.mark.parametrize("workspace", [True, False])
@pytest.mark.parametrize("specs", [
    # rows of different lengths in one launch, the longest last: cut into ranges of K beside a
    # problem that is stored directly, and (without a workspace, or too long for ranges) windows
    [(5, 48, 640, "fp16", 4, 0), (5, 272, 4224, "fp16", 4, 0), (5, 48, 14464, "fp16", 4, 0)],
    [(5, 48, 640, "bf16", 4, 0), (5, 272, 4224, "bf16", 4, 0), (5, 48, 14464, "bf16", 4, 0)],
    [(16, 48, 640, "bf16", 4, 0), (16, 80, 4224, "bf16", 4, 0)],
    [(16, 48, 640, "fp16", 8, 0), (16, 80, 4224, "fp16", 8, 0), (3, 16, 14464, "fp16", 8, 0)],
    # a problem with outliers beside one without
    [(5, 48, 640, "fp16", 4, 300), (5, 272, 4224, "fp16", 4, 0)],
    [(16, 48, 640, "bf16", 4, 300), (16, 48, 4224, "bf16", 4, 0), (16, 48, 640, "bf16", 4, 0)],
    # both activation types and code widths in one call: four launches share the workspace
    [(16, 48, 4224, "fp16", 4, 0), (16, 48, 4224, "bf16", 4, 0), (16, 48, 4224, "fp16", 8, 0),
     (16, 48, 4224, "bf16", 8, 0), (7, 272, 640, "fp16", 4, 0)],
])
def test_problems_of_different_kinds_streamed(specs, workspace):
    run_problems(specs, workspace)


@pytest.mark.parametrize("workspace", [True, False])
@pytest.mark.parametrize("specs", [
    # both paths in one call
    [(3, 272, 640, "bf16", 4, 0), (40, 272, 640, "bf16", 4, 0), (16, 48, 640, "bf16", 4, 0),
     (130, 48, 1152, "bf16", 4, 0)],
    # tiled launches with a problem that is split beside one that is not (one group of K)
    [(40, 48, 4224, "fp16", 4, 0), (130, 272, 128, "fp16", 4, 0), (17, 16, 4224, "fp16", 4, 0)],
    [(40, 48, 4224, "bf16", 8, 0), (130, 272, 128, "bf16", 8, 0), (17, 16, 4224, "bf16", 8, 0)],
    # outliers in one problem of a tiled launch, and a change of type and width in the middle
    [(40, 48, 640, "fp16", 4, 0), (40, 272, 640, "fp16", 4, 900), (70, 48, 640, "fp16", 4, 0),
     (70, 48, 640, "bf16", 4, 0), (40, 48, 640, "fp16", 8, 0), (40, 48, 640, "fp16", 4, 0)],
])
def test_problems_of_different_kinds_tiled(specs, workspace):
    run_problems(specs, workspace)


@pytest.mark.parametrize("M", [3, 40])
def test_more_problems_than_a_launch_holds(M):
    """Eleven problems: a second launch takes the last three, with their own epilogues."""
    run_problems([(M, 16 * (i + 1), 128 * (1 + i % 4), "fp16", 4, 0) for i in range(11)])


def test_empty_batch():
    torch = torch_cuda()
    w = weight(1, 48, 384)
    X = torch.empty((0, 384), dtype=torch.float16, device="cuda")
    assert tuple(w4.w4a16_linear(X, w.pw).shape) == (0, 48)
    assert tuple(w4.w4a16_gated(X, w.pw, w.pw).shape) == (0, 48)
    wt = w4.w4a16_transpose(w.pw)
    dX, dZ, db = w4.w4a16_linear_backward(torch.empty((0, 48), dtype=torch.float16, device="cuda"), wt,
                                          bias_grad=True)
    assert tuple(dX.shape) == (0, 384) and not values(db).any()
    e = torch.empty((0, 48), dtype=torch.float16, device="cuda")
    out = w4.w4a16_gated_backward(e, e, e, wt, wt, bias_grad=True)
    assert not values(out[3]).any() and not values(out[4]).any()


def test_extreme_pre_activations():
    """Large, infinite and NaN biases: the activations' limits, NaN kept as NaN."""
    torch = torch_cuda()
    N, K, M = 48, 384, 20
    w = weight(1, N, K)
    X, Xv = act_array("bf16", 1, M, K)
    big = np.zeros(N, np.float32)
    big[:8] = [1e38, -1e38, 1e20, -1e20, 300.0, -300.0, np.nan, 20.0]
    b = to_dev(to_bf16_bits(big).view(np.int16)).view(torch.bfloat16)
    bv = bf16_bits_to_f64(to_bf16_bits(big))
    for act in of.ACTS[1:]:
        for m in (M, 3):
            note(f"extreme pre-activations {act} M={m}")
            got = values(w4.w4a16_linear(X[:m], w.pw, bias=b, act=ACT[act]))
            z = Xv[:m] @ w.W.T + bv
            assert np.isnan(got[:, 6]).all()
            up, down = [0, 2, 4, 7], [1, 3, 5]
            tol = 2 * U["bf16"]
            assert (np.abs(got[:, up] - z[:, up]) <= tol * np.abs(z[:, up]) + 1.0 * (act != "relu") * 1e-6).all()
            assert (np.abs(got[:, down]) <= 1e-30).all()


# Pre-activations from far in the lower tail on, where an activation is all tail: past them
# its values leave the normal range of fp32 (and bf16).
TAIL = {"silu": -80.0, "gelu": -12.5, "gelu_tanh": -9.4}


def tail_points(dtype, act, n):
    """n pre-activations from the tail to 6: (device tensor [n], fp64 values)."""
    torch = torch_cuda()
    z = np.linspace(TAIL[act], 6.0, n).astype(np.float32)
    if dtype == "fp16":
        return to_dev(z.astype(np.float16)), z.astype(np.float16).astype(np.float64)
    b = to_bf16_bits(z)
    return to_dev(b.view(np.int16)).view(torch.bfloat16), bf16_bits_to_f64(b)


def tail_eps(z, act):
    """Relative error of the activation's factor (sigmoid or normal distribution function) in
    fp32: 2^-19 for its dozen roundings and the fits, reciprocal and exponential (at most
    2^-21 each), and the exponential's argument a, which a relative rounding of k 2^-24 moves by
    k |a| 2^-24: z^2 / 2 (one rounding, one more in the change of base), z (one), and
    sqrt(8 / pi) (z + 0.044715 z^3) (four)."""
    a = {"silu": np.abs(z), "gelu": z * z / 2,
         "gelu_tanh": 1.6 * np.abs(z + 0.044715 * z ** 3)}[act]
    return 2.0 ** -19 + a * (8 if act == "gelu_tanh" else 4) * 2.0 ** -24


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("M", [3, 40])
@pytest.mark.parametrize("act", list(TAIL))
def test_activations_keep_their_relative_precision(act, M, dtype):
    """X = 0, so Z is the bias without a rounding: Y (and H with U = 1) within one rounding of
    act(Z), relative to act(Z) itself."""
    torch = torch_cuda()
    N, K = 1008, 128
    note(f"tail of {act} M={M} {dtype}")
    w = weight(1, N, K)
    b, z = tail_points(dtype, act, N)
    X = torch.zeros(M, K, dtype=b.dtype, device="cuda")
    ref, u = of.act(z, act), U[dtype]
    bound = (u + 2 * tail_eps(z, act)) * np.abs(ref) + (TINY if dtype == "fp16" else 0.0)
    for got in (w4.w4a16_linear(X, w.pw, bias=b, act=ACT[act]),
                w4.w4a16_gated(X, w.pw, w.pw, act=ACT[act], bias_gate=b, bias_up=torch.ones_like(b))):
        bad = np.abs(values(got) - ref) > bound
        assert not bad.any(), (z[np.nonzero(bad)[1][:4]], (np.abs(values(got) - ref) / np.abs(ref)).max())


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("act", list(TAIL))
def test_derivatives_keep_their_relative_precision(act, dtype):
    """dZ of dY = 1 in the tail: act' = f + z f' with the factor f and its derivative, each to
    the factor's relative error (f' = f (1 - f) u' too, where 1 - f is within 2^-23)."""
    torch = torch_cuda()
    N, K, M = 1008, 128, 3
    note(f"tail of {act}' {dtype}")
    wt = w4.w4a16_transpose(weight(1, N, K).pw)
    zt, z = tail_points(dtype, act, N)
    Z = zt.expand(M, N).contiguous()
    dZ, one = torch.empty_like(Z), torch.ones_like(Z)
    w4.LinearBackwardCall([w4.BackwardTerm(one, wt, ACT[act], Z, dZ)], None, None)()
    ref, u = of.act_grad(z, act), U[dtype]
    f = of.act(z, act) / np.where(z == 0, 1.0, z)
    size = f + np.abs(ref - f) + np.abs(z) * f * {"silu": 1.0, "gelu": 0.0, "gelu_tanh":
                                                  1.6 * (1 + 3 * 0.044715 * z * z)}[act]
    bound = u * np.abs(ref) + 2 * tail_eps(z, act) * size + (TINY if dtype == "fp16" else 0.0)
    bad = np.abs(values(dZ) - ref) > bound
    assert not bad.any(), (z[np.nonzero(bad)[1][:4]], (np.abs(values(dZ) - ref) / bound).max())


EXTREMES = np.array([1e38, -1e38, 1e20, -1e20, 300.0, -300.0, 90.0, -90.0, 16.1, -16.1, 15.9, -15.9,
                     np.inf, -np.inf, np.nan, 0.0], np.float32)


def extreme_values(dtype, n):
    """n values that cycle through EXTREMES (fp16: large ones become infinite)."""
    torch = torch_cuda()
    z = np.resize(EXTREMES, n)
    if dtype == "fp16":
        with np.errstate(over="ignore"):
            h = z.astype(np.float16)
        return to_dev(h), h.astype(np.float64)
    b = to_bf16_bits(z)
    return to_dev(b.view(np.int16)).view(torch.bfloat16), bf16_bits_to_f64(b)


def check_extreme_act(got, z, dtype, act):
    """act(z) at its limits: z or 0 to either side of 15; NaN stays NaN.  At minus infinity the
    formulas are infinity times 0: 0 or NaN (relu: 0)."""
    assert np.isnan(got[:, np.isnan(z)]).all()
    up, down = z > 15, (z < -15) & np.isfinite(z)
    # products with U = 1, sums with X = 0: one rounding of z, past the limit 1e-6 from gelu_tanh's factor
    with np.errstate(invalid="ignore"):
        near = np.abs(got[:, up] - z[up]) <= (U[dtype] + 1e-6) * np.abs(z[up])
    assert (near | (got[:, up] == z[up])).all()
    assert (np.abs(got[:, down]) <= (5e-6 if act == "silu" else 1e-30)).all()
    assert (got[:, z == 0] == 0).all()
    low = got[:, z == -np.inf]
    assert ((low == 0) | (np.isnan(low) & (act != "relu"))).all()


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("M,K", [(3, 384), (20, 384), (5, 14464), (20, 4224)])
@pytest.mark.parametrize("act", of.ACTS[1:])
def test_activations_at_their_limits(act, M, K, dtype):
    """Large, infinite and NaN pre-activations (X = 0 and such a bias), direct and out of K
    ranges and split sums, in a linear and in a gated call."""
    torch = torch_cuda()
    N = 48
    w = weight(1, N, K)
    b, z = extreme_values(dtype, N)
    X = torch.zeros(M, K, dtype=b.dtype, device="cuda")
    note(f"limits of {act} M={M} K={K} {dtype}")
    check_extreme_act(values(w4.w4a16_linear(X, w.pw, bias=b, act=ACT[act])), z, dtype, act)
    check_extreme_act(values(w4.w4a16_gated(X, w.pw, w.pw, act=ACT[act], bias_gate=b,
                                            bias_up=torch.ones_like(b))), z, dtype, act)


# ---- backward -----------------------------------------------------------------------

def eval_bound(dY, z, extra=0.0):
    return 2.0 ** -18 * np.abs(dY) * (1 + np.abs(z)) * (1 + extra)


def dx_bound(dZs, Ds, s, u, Ntot, ref, e_dZs):
    b = 0.0
    for d, D, e in zip(dZs, Ds, e_dZs):
        b = b + (2 * u + 2 * u * u + (Ntot + 8) * 2.0 ** -24) * (np.abs(d) @ np.abs(D)) \
            + (e + TINY) @ np.abs(D)
    return (b if s is None else b * s.astype(np.float64)) * (1 + u) + u * np.abs(ref) + TINY


def run_linear_backward(M, N, K, dtype, act="none", add=False, bias=False, awq=False, bits=4,
                        inplace=False):
    torch = torch_cuda()
    note(f"linear backward M={M} N={N} K={K} {dtype} {act} add={add} bias={bias} awq={awq} bits={bits} "
         f"inplace={inplace}")
    w = weight(6, N, K, awq, bits)
    wt = w4.w4a16_transpose(w.pw)
    dY, dYv = act_array(dtype, 11, M, N, 0.25)
    Z, Zv = act_array(dtype, 12, M, N)
    dX, buf = guarded(dtype, M, K)
    A, Av = act_array(dtype, 13, M, K) if add else (None, None)
    if inplace and add:
        dX.copy_(A)
        A = dX
    dZ, zbuf = guarded(dtype, M, N)
    if act == "none":
        Z, dZ = None, None
    elif inplace:
        dZ = Z if M % 2 else dY
    db = torch.full((N,), float("nan"), device="cuda") if bias else None
    w4.LinearBackwardCall([w4.BackwardTerm(dY, wt, ACT[act], Z, dZ, db)], w.sd, dX, A)()
    dz = of.linear_grad(dYv, Zv, act)
    ref = of.input_grad([dz], [w.W], Av)
    u, tag = U[dtype], f"backward {M}x{N}x{K} {dtype}"
    e = eval_bound(dYv, Zv) if act != "none" else np.zeros_like(dYv)
    check_guard(buf, M)
    if act != "none":
        close(values(dZ), dz, u * np.abs(dz) + e + TINY, tag + " dZ", REL[dtype])
        check_guard(zbuf, M)
    close(values(dX), ref, dx_bound([dz], [w.D], w.s, u, N, ref, [e]), tag, REL[dtype])
    if bias:
        bound = (M + 8) * 2.0 ** -24 * np.abs(dz).sum(0) + e.sum(0) + 1e-30
        assert (np.abs(values(db) - dz.sum(0)) <= bound).all(), tag + " dbias"


def run_gated_backward(M, N, K, dtype, act="silu", add=False, bias=False, awq=False, bits=4,
                       inplace=False):
    torch = torch_cuda()
    note(f"gated backward M={M} N={N} K={K} {dtype} {act} add={add} bias={bias} awq={awq} bits={bits} "
         f"inplace={inplace}")
    wg, wu = weight(6, N, K, awq, bits), weight(8, N, K, awq, bits)
    gt, ut = w4.w4a16_transpose(wg.pw), w4.w4a16_transpose(wu.pw)
    dH, dHv = act_array(dtype, 11, M, N, 0.25)
    G, Gv = act_array(dtype, 12, M, N)
    Up, Uv = act_array(dtype, 14, M, N)
    dX, buf = guarded(dtype, M, K)
    A, Av = act_array(dtype, 13, M, K) if add else (None, None)
    dG, gbuf = guarded(dtype, M, N)
    dU, ubuf = guarded(dtype, M, N)
    if inplace:
        dG, dU = G, Up
    db = [torch.full((N,), float("nan"), device="cuda") if bias else None for _ in range(2)]
    w4.GatedBackwardCall(dH, G, Up, gt, ut, wg.sd, dX, dG, dU, ACT[act], A, *db)()
    dg, du = of.gated_grad(dHv, Gv, Uv, act)
    ref = of.input_grad([dg, du], [wg.W, wu.W], Av)
    u, tag = U[dtype], f"gated backward {M}x{N}x{K} {dtype}"
    e = eval_bound(dHv, Gv, np.abs(Uv))
    check_guard(buf, M), check_guard(gbuf, M), check_guard(ubuf, M)
    close(values(dG), dg, u * np.abs(dg) + e + TINY, tag + " dG", REL[dtype])
    close(values(dU), du, u * np.abs(du) + e + TINY, tag + " dU", REL[dtype])
    close(values(dX), ref, dx_bound([dg, du], [wg.D, wu.D], wg.s, u, 2 * N, ref, [e, e]), tag, REL[dtype])
    if bias:
        for t, d in zip(db, (dg, du)):
            bound = (M + 8) * 2.0 ** -24 * np.abs(d).sum(0) + e.sum(0) + 1e-30
            assert (np.abs(values(t) - d.sum(0)) <= bound).all(), tag + " dbias"


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("N,K", [(16, 128), (128, 128), (144, 384), (272, 640), (528, 1152)])
def test_transposed_copy_is_exact(N, K, bits):
    note(f"transpose N={N} K={K} bits={bits}")
    w = weight(6, N, K, False, bits)
    wt = w4.w4a16_transpose(w.pw)
    assert np.array_equal(to_host(wt.wt), of.transpose_codes(w.q, bits))
    got = to_host(wt.meta).view(np.uint16)
    assert np.array_equal(got, of.transpose_meta(w.scales, w.zeros, bits).view(np.uint16))


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("M", [1, 3, 16, 17, 32, 33, 64, 65, 129, 300])
def test_linear_backward_every_tile_height(M, dtype):
    run_linear_backward(M, 272, 640, dtype, "gelu", add=True, bias=True, awq=M % 2 == 1)


@pytest.mark.parametrize("act", of.ACTS)
def test_linear_backward_activations(act):
    run_linear_backward(40, 48, 384, "fp16", act, bias=True)
    run_linear_backward(40, 48, 384, "bf16", act, add=True)


@pytest.mark.parametrize("M,N,K", [(1, 16, 128), (20, 16, 256), (70, 16, 128), (5, 14336, 128),
                                   (64, 18944, 256), (100, 4096, 384), (1, 48, 14336), (257, 144, 2048)])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_linear_backward_extreme_shapes(M, N, K, dtype):
    run_linear_backward(M, N, K, dtype, "none", add=True, bias=True, awq=True)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("M", [31, 128, 129, 256, 257])
def test_bias_gradients_around_the_one_strip_limit(M, dtype):
    """Column blocks in part (80 and 528 columns) on both sides of where one strip holds all rows."""
    run_linear_backward(M, 80, 256, dtype, "none", bias=True)
    run_linear_backward(M, 528, 128, dtype, "silu", bias=True, inplace=True)
    run_gated_backward(M, 80, 128, dtype, "gelu_tanh", bias=True)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("M", [1, 20, 40, 100, 200])
def test_backward_int8_codes(M, dtype):
    run_linear_backward(M, 272, 640, dtype, "silu", add=True, bias=True, awq=True, bits=8)
    run_gated_backward(M, 144, 384, dtype, "silu", add=True, bias=True, bits=8)


@pytest.mark.parametrize("M", [9, 40, 130])
def test_backward_in_place(M):
    run_linear_backward(M, 272, 640, "bf16", "silu", add=True, inplace=True)
    run_linear_backward(M, 1040, 256, "fp16", "gelu", add=True, bias=True, inplace=True)
    run_gated_backward(M, 272, 640, "bf16", "gelu", bias=True, inplace=True)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("M", [3, 300])
@pytest.mark.parametrize("act", of.ACTS[1:])
def test_derivatives_at_their_limits(act, M, dtype):
    """act' is 1 above and 0 below the middle, without a NaN from a vanishing factor times an
    overflowed one; NaN stays NaN, and at the infinities silu's and gelu's formulas are infinity
    times 0 (1, 0 or NaN)."""
    torch = torch_cuda()
    N, K = 48, 128
    wt = w4.w4a16_transpose(weight(1, N, K).pw)
    zt, z = extreme_values(dtype, N)
    Z = zt.expand(M, N).contiguous()
    one = torch.ones_like(Z)
    note(f"limits of {act}' M={M} {dtype}")
    dZ, dG, dU = torch.empty_like(Z), torch.empty_like(Z), torch.empty_like(Z)
    w4.LinearBackwardCall([w4.BackwardTerm(one, wt, ACT[act], Z, dZ)], None, None)()
    w4.GatedBackwardCall(one, Z, one, wt, wt, None, None, dG, dU, ACT[act])()
    got = values(dZ)
    assert np.array_equal(got, values(dG), equal_nan=True)
    check_extreme_act(values(dU), z, dtype, act)                 # dU = dH act(G)
    assert np.isnan(got[:, np.isnan(z)]).all()
    up, down = (z > 15) & np.isfinite(z), (z < -15) & np.isfinite(z)
    assert (np.abs(got[:, up] - 1) <= U[dtype] + 1e-5).all()
    assert (np.abs(got[:, down]) <= (5e-6 if act == "silu" else 1e-30)).all()
    for inf, limit in ((np.inf, 1.0), (-np.inf, 0.0)):
        at = got[:, z == inf]
        assert ((at == limit) | (np.isnan(at) & (act in ("silu", "gelu")))).all()


@pytest.mark.parametrize("M", [9, 130, 300])
def test_gated_backward_into_dH(M):
    """dG, or dU, written where dH is: the bits of the call with buffers of their own."""
    torch = torch_cuda()
    N, K = 272, 640
    gt, ut = (w4.w4a16_transpose(weight(k, N, K).pw) for k in (6, 8))
    G, Up = act_array("bf16", 12, M, N)[0], act_array("bf16", 14, M, N)[0]
    dH = act_array("bf16", 11, M, N, 0.25)[0]
    want = w4.w4a16_gated_backward(dH, G, Up, gt, ut, bias_grad=True)
    for which in (0, 1):
        d, other, dX = dH.clone(), torch.empty_like(dH), torch.empty_like(want[0])
        db = [torch.empty(N, device="cuda") for _ in range(2)]
        note(f"gated backward into dH M={M} output {which}")
        outs = (d, other) if which == 0 else (other, d)
        w4.GatedBackwardCall(d, G, Up, gt, ut, None, dX, *outs, w4.ACT_SILU, None, *db)()
        for a, b in zip(want, (dX, *outs, *db)):
            assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("M", [1, 3, 16, 17, 33, 65, 129, 300])
def test_gated_backward_every_tile_height(M, dtype):
    run_gated_backward(M, 272, 640, dtype, "silu", add=M % 2 == 0, bias=True, awq=M % 2 == 1)


@pytest.mark.parametrize("act", of.ACTS)
def test_gated_backward_activations(act):
    run_gated_backward(40, 48, 384, "fp16", act, bias=True)
    run_gated_backward(40, 48, 384, "bf16", act, add=True)


@pytest.mark.parametrize("M,N,K", [(1, 16, 128), (70, 16, 128), (64, 9472, 256), (200, 2064, 128)])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_gated_backward_extreme_shapes(M, N, K, dtype):
    run_gated_backward(M, N, K, dtype, "silu", add=True, bias=True, awq=True)


@pytest.mark.parametrize("M", [5, 40, 140])
def test_backward_rows_are_independent(M):
    """NaN and infinities in one row of dY reach no other row, ragged N included: the
    chunks past N of the row before must read as zeros, not as that row."""
    torch = torch_cuda()
    N, K = 144, 384
    w = weight(6, N, K)
    wt = w4.w4a16_transpose(w.pw)
    dY, dYv = act_array("bf16", 11, M, N, 0.25)
    clean = values(w4.w4a16_linear_backward(dY, wt)[0])
    for row in (1, M - 1):
        bad = dY.clone()
        bad[row] = float("nan")
        bad[row, 0] = float("inf")
        note(f"backward row independence M={M} row={row}")
        got = values(w4.w4a16_linear_backward(bad, wt)[0])
        keep = np.arange(M) != row
        assert np.array_equal(got[keep], clean[keep])
        assert np.isnan(got[row]).all()


@pytest.mark.parametrize("M", [17, 100])
def test_backward_of_several_layers(M):
    """q, k and v read one X: dX is the sum of their products, the same weight twice too."""
    torch = torch_cuda()
    K, dtype = 640, "fp16"
    for Ns in ((272,), (272, 48, 16), (144, 144), (16, 528, 48, 272)):
        terms, dzs, Ws, Ds, es = [], [], [], [], []
        for i, N in enumerate(Ns):
            w = weight(6 + 10 * (N != 144) * i, N, K)
            act = ("none", "silu")[i % 2]
            dY, dYv = act_array(dtype, 50 + i, M, N, 0.25)
            Z, Zv = act_array(dtype, 60 + i, M, N)
            dZ = torch.empty_like(dY) if act != "none" else None
            db = torch.empty(N, device="cuda") if i != 1 else None
            terms.append(w4.BackwardTerm(dY, w4.w4a16_transpose(w.pw), ACT[act],
                                         Z if dZ is not None else None, dZ, db))
            dzs.append(of.linear_grad(dYv, Zv, act))
            es.append(eval_bound(dYv, Zv))
            Ws.append(w.W)
            Ds.append(w.D)
        dX = torch.empty((M, K), dtype=torch.float16, device="cuda")
        note(f"backward of layers {Ns} M={M}")
        w4.LinearBackwardCall(terms, None, dX)()
        ref = of.input_grad(dzs, Ws)
        close(values(dX), ref, dx_bound(dzs, Ds, None, U[dtype], sum(Ns), ref, es), f"{Ns}", REL[dtype])
        for t, d, e in zip(terms, dzs, es):
            if t.dbias is not None:
                assert (np.abs(values(t.dbias) - d.sum(0))
                        <= (M + 8) * 2.0 ** -24 * np.abs(d).sum(0) + e.sum(0) + 1e-30).all()


def test_backward_without_dx():
    torch = torch_cuda()
    M, N, K = 50, 272, 640
    wt = w4.w4a16_transpose(weight(6, N, K).pw)
    dY, dYv = act_array("bf16", 11, M, N)
    db = torch.empty(N, device="cuda")
    w4.LinearBackwardCall([w4.BackwardTerm(dY, wt, dbias=db)], None, None)()
    assert (np.abs(values(db) - dYv.sum(0)) <= (M + 8) * 2.0 ** -24 * np.abs(dYv).sum(0) + 1e-30).all()


def test_linear_past_32_bit_offsets():
    """X and Y of more than 2^31 bytes: rows at the start, around the 2 GiB offsets and at the
    end against the oracle."""
    torch = torch_cuda()
    M, N, K = 270_001, 4096, 4096
    note(f"linear M={M} N={N} K={K}: X and Y past 2 GiB")
    w = weight(30, N, K)
    X = torch.randn(M, K, device="cuda", generator=torch.Generator("cuda").manual_seed(3)).half()
    R = X.flip(0).contiguous()
    Y = w4.w4a16_linear(X, w.pw, residual=R, act=w4.ACT_RELU)
    rows = torch.tensor([0, 1, 131071, 131072, 262143, 262144, 262145, M - 2, M - 1])
    Xv = values(X[rows.cuda()])
    ref, z = of.linear(Xv, w.W, None, "relu", values(R[rows.cuda()]))
    e = act_bound(z, product_bound(Xv, w.W, U["fp16"], K))
    close(values(Y[rows.cuda()]), ref, e + U["fp16"] * (np.abs(ref) + e) + TINY, "large", 5 * REL["fp16"])


def test_backward_past_32_bit_offsets():
    torch = torch_cuda()
    M, N, K = 270_001, 4112, 128
    note(f"backward M={M} N={N} K={K}: dY past 2 GiB")
    w = weight(31, N, K)
    dY = (torch.randn(M, N, device="cuda", generator=torch.Generator("cuda").manual_seed(4)) * 0.25).half()
    dX, dZ, db = w4.w4a16_linear_backward(dY, w4.w4a16_transpose(w.pw), bias_grad=True)
    rows = torch.tensor([0, 1, 130559, 130560, 261118, 261119, 261120, M - 2, M - 1])
    d = values(dY[rows.cuda()])
    ref = of.input_grad([d], [w.W])
    close(values(dX[rows.cuda()]), ref,
          dx_bound([d], [w.D], None, U["fp16"], N, ref, [np.zeros_like(d)]), "large", REL["fp16"])
    total, size = values(dY.double().sum(0)), values(dY.abs().double().sum(0))
    # at most (M / 256 rows + 4 lanes + 256 strips) additions in a row
    assert (np.abs(values(db) - total) <= (M / 256 + 260) * 2.0 ** -24 * size).all()


def test_binding_refuses_views_types_and_shapes():
    torch = torch_cuda()
    w = weight(1, 48, 384)
    X = torch.zeros(6, 384, dtype=torch.float16, device="cuda")
    b = torch.zeros(48, dtype=torch.float16, device="cuda")
    wt = w4.w4a16_transpose(w.pw)
    dY = torch.zeros(6, 48, dtype=torch.float16, device="cuda")
    for bad, kw in ((X[::2], {}), (X.t().contiguous().t(), {}), (X[:, :256], {}), (X[None], {})):
        with pytest.raises(ValueError):
            w4.w4a16_linear(bad, w.pw, **kw)
    for kw in (dict(bias=b[:32]), dict(residual=dY[:3]), dict(preact=dY.t().contiguous().t()),
               dict(out=torch.zeros(6, 64, dtype=torch.float16, device="cuda"))):
        with pytest.raises(ValueError):
            w4.w4a16_linear(X, w.pw, **kw)
    for kw in (dict(bias=b.float()), dict(bias=b.bfloat16()), dict(residual=dY.cpu()), dict(s=b.float())):
        with pytest.raises((TypeError, ValueError)):
            w4.w4a16_linear(X, w.pw, **kw)
    with pytest.raises(TypeError):
        w4.w4a16_linear(X.float(), w.pw)
    with pytest.raises(ValueError):
        w4.w4a16_gated(X, w.pw, weight(1, 272, 640).pw)
    with pytest.raises(ValueError):
        w4.w4a16_linear_backward(dY[:, ::2], wt)
    with pytest.raises(ValueError):
        w4.w4a16_linear_backward(dY, wt, act=w4.ACT_SILU, preact=dY[:3])
    with pytest.raises(w4.W4A16Error) as e:
        w4.w4a16_linear_backward(dY, wt, act=w4.ACT_SILU)            # no pre-activation
    assert e.value.status == -1
    with pytest.raises(w4.W4A16Error) as e:
        w4.w4a16_linear(X, w.pw, act=17)
    assert e.value.status == -3
    with pytest.raises(ValueError):
        w4.w4a16_transpose(weight(1, 272, 640, False, 4, 900).pw)    # fp16 outliers
    small = torch.zeros(16, dtype=torch.uint8, device="cuda")
    with pytest.raises(ValueError):
        w4.LinearCall([(torch.zeros(64, 4096, dtype=torch.float16, device="cuda"), weight(1, 16, 4096).pw,
                        None, torch.zeros(64, 16, dtype=torch.float16, device="cuda"), w4.Epilogue())],
                      workspace=small)


def test_tensors_that_require_grad():
    """Refused in grad mode, whichever it is; taken under no_grad and inside an
    autograd.Function, whose gradients are the formulas'."""
    torch = torch_cuda()
    N, K, M = 48, 384, 6
    w = weight(1, N, K)
    wt = w4.w4a16_transpose(w.pw)
    t = lambda *shape: torch.randn(*shape, generator=torch.Generator().manual_seed(5)).half().cuda()
    X, b, R, Y, s = t(M, K), t(N), t(M, N), t(M, N), t(K).abs() + 0.5
    for name, base in (("bias", b), ("residual", R), ("preact", Y), ("out", Y), ("s", s)):
        with pytest.raises(ValueError, match="requires grad"):
            w4.w4a16_linear(X, w.pw, **{name: base.clone().requires_grad_()})
    for name in ("bias_gate", "bias_up"):
        with pytest.raises(ValueError, match="requires grad"):
            w4.w4a16_gated(X, w.pw, w.pw, **{name: b.clone().requires_grad_()})
    with pytest.raises(ValueError, match="requires grad"):
        w4.w4a16_linear_backward(R, wt, act=w4.ACT_SILU, preact=Y.clone().requires_grad_())
    with pytest.raises(ValueError, match="requires grad"):
        w4.w4a16_gated_backward(R, Y, Y.clone().requires_grad_(), wt, wt)

    class Layer(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, bias):
            z = torch.empty(M, N, dtype=x.dtype, device="cuda")
            ctx.save_for_backward(z)
            return w4.w4a16_linear(x, w.pw, bias=bias, act=w4.ACT_SILU, preact=z)

        @staticmethod
        def backward(ctx, dy):
            dX, _, db = w4.w4a16_linear_backward(dy.contiguous(), wt, act=w4.ACT_SILU,
                                                 preact=ctx.saved_tensors[0], bias_grad=True)
            return dX, db.half()
    note("autograd.Function of a layer")
    x, bias = X.clone().requires_grad_(), b.clone().requires_grad_()
    Layer.apply(x, bias).backward(R)
    with torch.no_grad():
        assert torch.equal(Layer.apply(x, bias), w4.w4a16_linear(x, w.pw, bias=bias, act=w4.ACT_SILU))
    z = values(X) @ w.W.T + values(b)
    dz = of.linear_grad(values(R), z, "silu")
    # z is rounded once before its derivative, dZ once before the product
    assert errors(values(x.grad), of.input_grad([dz], [w.W]))[0] <= 5 * REL["fp16"]
    assert errors(values(bias.grad), dz.sum(0))[0] <= 5 * REL["fp16"]


# ---- together -----------------------------------------------------------------------

@pytest.mark.parametrize("M", [5, 70])
def test_feed_forward_block_and_its_gradient(M):
    """A whole block, forward and backward, as a training step calls it: out = X + down(
    silu(gate X) * up X), against the oracle's formulas and a directional difference."""
    torch = torch_cuda()
    K, N, dtype = 384, 272 - 16, "fp16"       # the down projection reads N = 256 columns
    wg, wu, wd = weight(2, N, K), weight(4, N, K), weight(6, K, N)
    X, Xv = act_array(dtype, 1, M, K)
    G, Up = torch.empty((2, M, N), dtype=torch.float16, device="cuda")
    note(f"feed-forward block M={M}")
    H = w4.w4a16_gated(X, wg.pw, wu.pw, preact=(G, Up))
    out = w4.w4a16_linear(H, wd.pw, residual=X)
    dO, dOv = act_array(dtype, 70, M, K)
    dH = w4.w4a16_linear_backward(dO, w4.w4a16_transpose(wd.pw))[0]
    dX, dG, dU, _, _ = w4.w4a16_gated_backward(dH, G, Up, w4.w4a16_transpose(wg.pw),
                                               w4.w4a16_transpose(wu.pw), add=dO)

    def block(x):
        h, g, u = of.gated(x, wg.W, wu.W)
        return of.linear(h, wd.W, residual=x)[0], g, u
    ref, g, u = block(Xv)
    # H carries 5 x REL, the down product REL more
    assert errors(values(out) - Xv, ref - Xv)[0] <= 8 * REL[dtype]
    dh = of.input_grad([dOv], [wd.W])
    dg, du = of.gated_grad(dh, g, u)
    dx = of.input_grad([dg, du], [wg.W, wu.W], dOv)
    for got, want in ((dG, dg), (dU, du), (dX, dx)):
        assert errors(values(got), want)[0] <= 8 * REL[dtype]
    v = np.random.default_rng(9).standard_normal((M, K))
    h = 1e-5
    num = ((block(Xv + h * v)[0] - block(Xv - h * v)[0]) * dOv).sum() / (2 * h)
    # the directional derivative: Cauchy-Schwarz on the relative L2 bound of dX
    assert abs((values(dX) * v).sum() - num) <= 8 * REL[dtype] * np.linalg.norm(dx) * np.linalg.norm(v)


def _step(M, K, N, dtype="bf16"):
    """Prepared calls of a block's forward and backward over fixed buffers."""
    torch = torch_cuda()
    dt = torch.bfloat16 if dtype == "bf16" else torch.float16
    wg, wu, wd = weight(2, N, K), weight(4, N, K), weight(6, K, N)
    X, dO = act_array(dtype, 1, M, K)[0], act_array(dtype, 70, M, K)[0]
    e = lambda *s, d=dt: torch.zeros(*s, dtype=d, device="cuda")
    H, G, Up, out, dH, dG, dU, dX = (e(M, N), e(M, N), e(M, N), e(M, K), e(M, N), e(M, N), e(M, N),
                                     e(M, K))
    db = e(N, d=torch.float32)
    tg, tu, td = (w4.w4a16_transpose(w.pw) for w in (wg, wu, wd))
    calls = [w4.GatedCall(X, wg.pw, wu.pw, None, H, preact=(G, Up)),
             w4.LinearCall([(H, wd.pw, None, out, w4.Epilogue(residual=X))]),
             w4.LinearBackwardCall([w4.BackwardTerm(dO, td)], None, dH),
             w4.GatedBackwardCall(dH, G, Up, tg, tu, None, dX, dG, dU, add=dO, dbias_gate=db)]
    return calls, (H, G, Up, out, dH, dG, dU, dX, db), (X, dO)


@pytest.mark.parametrize("M", [3, 64, 200])
def test_captured_and_replayed(M):
    """A captured step replayed with eager work between the replays: the eager bits each
    time, with new inputs too."""
    torch = torch_cuda()
    calls, outs, (X, dO) = _step(M, 640, 1152)

    def run():
        for c in calls:
            c()
    note(f"capture M={M}")
    run()
    want = [values(t) for t in outs]
    g = torch.cuda.CUDAGraph()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st), torch.cuda.graph(g, stream=st):
        run()
    for rep in range(3):
        for t in outs:
            t.fill_(float("nan"))
        g.replay()
        for a, b in zip(want, [values(t) for t in outs]):
            assert np.array_equal(a, b), rep
        run()                                  # eager work between the replays
        torch.cuda.synchronize()
    X.copy_(X.flip(0).clone())
    dO.copy_(dO.flip(0).clone())
    g.replay()
    got = [values(t) for t in outs]
    run()
    for a, b in zip(got, [values(t) for t in outs]):
        assert np.array_equal(a, b)


def test_two_streams_at_once():
    """Two steps with workspaces of their own on two streams, nothing between them."""
    torch = torch_cuda()
    a, b = _step(64, 640, 1152), _step(40, 1152, 640)
    want = []
    for calls, outs, _ in (a, b):
        for c in calls:
            c()
        want.append([values(t) for t in outs])
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    note("two streams")
    for rep in range(5):
        for i in range(4):
            for st, (calls, _, _) in zip(s, (a, b)):
                with torch.cuda.stream(st):
                    calls[i]()
        torch.cuda.synchronize()
        for w, (_, outs, _) in zip(want, (a, b)):
            for x, t in zip(w, outs):
                assert np.array_equal(x, values(t)), rep


@pytest.mark.parametrize("M", [1, 16, 48, 130])
def test_same_bits_every_time(M):
    calls, outs, _ = _step(M, 1152, 528 - 16)
    runs = []
    for _ in range(3):
        for c in calls:
            c()
        runs.append([values(t) for t in outs])
    for r in runs[1:]:
        for a, b in zip(runs[0], r):
            assert np.array_equal(a, b)


def test_plain_epilogue_gives_the_plain_products_bits():
    """No bias, activation or residual on the streaming path (M <= 16), where both calls
    split K alike: w4a16_linear is w4a16_gemm, bit for bit."""
    torch = torch_cuda()
    for dtype in ("fp16", "bf16"):
        for M in (1, 5, 16):
            w = weight(1, 272, 640, True)
            X, _ = act_array(dtype, 1, M, 640)
            note(f"plain epilogue {dtype} M={M}")
            assert torch.equal(w4.w4a16_linear(X, w.pw, w.sd), w4.w4a16_gemm(X, w.pw, w.sd))
