"""Refusals of the fused layers' entry points (host validation, no GPU), their sizes, and
the registers of the new kernels."""
import ctypes

import pytest

import weight_only_int4_group_amd as w4
from tests.test_kernel_sources import _device_asm, _kernel_metadata

V = ctypes.c_void_p
A, B = 1 << 20, 1 << 21           # aligned stand-in addresses (never dereferenced)
ODD = (1 << 20) + 2


def problem(**kw):
    f = dict(X=A, Wq=A, scales=A, zeros=A, s=None, Y=A, M=1, N=16, K=128, o_row_ptr=None, o_col=None,
             o_val=None, dtype=0, wbits=4)
    f.update(kw)
    return w4.Problem(*f.values())


def epilogue(bias=None, residual=None, preact=None, act=0):
    return w4.EpilogueStruct(bias, residual, preact, act)


def linear_rc(p, e, count=1, ws=None, nbytes=0):
    return w4.lib().w4a16_linear(ctypes.byref(p) if p else None, ctypes.byref(e) if e else None, count,
                                 ws, nbytes, None)


@pytest.mark.parametrize("pk,ek,code", [
    (dict(K=100), {}, -1), (dict(N=8), {}, -1), (dict(X=None), {}, -1), (dict(Y=None), {}, -1),
    (dict(Y=ODD), {}, -2), (dict(dtype=2), {}, -3), (dict(wbits=5), {}, -3),
    ({}, dict(act=5), -3), ({}, dict(act=-1), -3), ({}, dict(bias=ODD), -2),
    ({}, dict(residual=ODD), -2), ({}, dict(preact=ODD), -2), (dict(M=-1), {}, -1),
    (dict(o_col=A), {}, -1),
])
def test_linear_refusals(pk, ek, code):
    assert linear_rc(problem(**pk), epilogue(**ek)) == code
    n = ctypes.c_size_t()
    assert w4.lib().w4a16_linear_workspace_size(ctypes.byref(problem(**pk)), ctypes.byref(epilogue(**ek)),
                                                1, ctypes.byref(n)) == code


def test_linear_arrays_and_workspace():
    p, e = problem(), epilogue()
    assert linear_rc(None, None, 0) == 0
    assert linear_rc(None, e) == -1 and linear_rc(p, None) == -1 and linear_rc(p, e, -1) == -1
    assert linear_rc(p, e, ws=ODD, nbytes=64) == -2
    assert linear_rc(problem(M=0, X=None, Y=None), e) == 0
    assert w4.lib().w4a16_linear_workspace_size(ctypes.byref(p), ctypes.byref(e), 1, None) == -1


def gated_rc(g=None, u=None, H=A, bg=None, bu=None, act=2, ws=None, nbytes=0):
    g, u = problem(**{"Y": None, **(g or {})}), problem(**{"Y": None, **(u or {})})
    return w4.lib().w4a16_gated(ctypes.byref(g), ctypes.byref(u), bg, bu, act, H, ws, nbytes, None)


@pytest.mark.parametrize("kw,code", [
    (dict(H=None), -1), (dict(H=ODD), -2), (dict(act=9), -3), (dict(bg=ODD), -2), (dict(bu=ODD), -2),
    (dict(u=dict(X=B)), -1), (dict(u=dict(s=A)), -1), (dict(u=dict(N=32)), -1), (dict(u=dict(K=256)), -1),
    (dict(u=dict(M=2)), -1), (dict(u=dict(dtype=1)), -1), (dict(u=dict(wbits=8)), -1),
    (dict(g=dict(Y=A)), -1), (dict(u=dict(Y=A)), -1), (dict(g=dict(Y=A), u=dict(Y=ODD)), -2),
    (dict(g=dict(Wq=None)), -1), (dict(u=dict(scales=ODD)), -2), (dict(ws=ODD, nbytes=8), -2),
    (dict(g=dict(K=100), u=dict(K=100)), -1),
])
def test_gated_refusals(kw, code):
    assert gated_rc(**kw) == code


def test_gated_null_and_empty():
    L = w4.lib()
    p = problem()
    assert L.w4a16_gated(None, ctypes.byref(p), None, None, 2, A, None, 0, None) == -1
    assert L.w4a16_gated_workspace_size(ctypes.byref(p), ctypes.byref(p), None) == -1
    assert gated_rc(g=dict(M=0, X=None), u=dict(M=0, X=None), H=None) == 0


@pytest.mark.parametrize("N,K,wbits,sizes", [
    (16, 128, 4, (128 * 64, 512)), (128, 256, 4, (128 * 128, 1024)), (144, 384, 4, (256 * 192, 2 * 3 * 512)),
    (144, 384, 8, (256 * 384, 2 * 3 * 512)), (14336, 4096, 0, (14336 * 2048, 112 * 32 * 512)),
])
def test_transposed_sizes(N, K, wbits, sizes):
    a, b = ctypes.c_size_t(), ctypes.c_size_t()
    assert w4.lib().w4a16_transposed_sizes(N, K, wbits, ctypes.byref(a), ctypes.byref(b)) == 0
    assert (a.value, b.value) == sizes


@pytest.mark.parametrize("N,K,wbits,code", [(0, 128, 4, -1), (16, 100, 4, -1), (24, 128, 4, -1),
                                            (16, 128, 3, -3), (1 << 23, 128, 4, -1),
                                            (16, 1 << 24, 8, -1), (65536, 65536, 4, -1)])
def test_transpose_refusals(N, K, wbits, code):
    a, b = ctypes.c_size_t(), ctypes.c_size_t()
    assert w4.lib().w4a16_transposed_sizes(N, K, wbits, ctypes.byref(a), ctypes.byref(b)) == code
    assert w4.lib().w4a16_transpose(A, A, A, N, K, wbits, A, A, None) == code
    for i in range(5):
        args = [A, A, A, 16, 128, 4, A, A, None]
        args[(0, 1, 2, 6, 7)[i]] = None
        assert w4.lib().w4a16_transpose(*args) == -1
        args[(0, 1, 2, 6, 7)[i]] = ODD
        assert w4.lib().w4a16_transpose(*args) == -2


def term(**kw):
    f = dict(dY=A, preact=A, dZ=A, dbias=None, Wt=A, meta=A, N=16, act=2, wbits=4)
    f.update(kw)
    return w4.BackwardTermStruct(*f.values())


def backward_rc(t=None, count=1, s=None, add=None, dX=A, M=1, K=128, dtype=0, ws=A, nbytes=1 << 30,
                terms=None):
    arr = (w4.BackwardTermStruct * max(count, 1))(*(terms or [term(**(t or {}))] * max(count, 1)))
    return w4.lib().w4a16_linear_backward(arr, count, s, add, dX, M, K, dtype, ws, nbytes, None)


@pytest.mark.parametrize("kw,code", [
    (dict(count=0), -1), (dict(count=5), -1), (dict(M=-1), -1), (dict(M=1 << 23), -1), (dict(K=100), -1),
    (dict(dtype=3), -3), (dict(t=dict(act=7)), -3), (dict(t=dict(wbits=6)), -3), (dict(t=dict(N=8)), -1),
    (dict(t=dict(N=1 << 23)), -1), (dict(t=dict(dY=None)), -1), (dict(t=dict(preact=None)), -1),
    (dict(t=dict(dZ=None)), -1), (dict(t=dict(act=0)), -1), (dict(t=dict(Wt=None)), -1),
    (dict(t=dict(meta=None)), -1), (dict(t=dict(dY=ODD)), -2), (dict(t=dict(dbias=ODD)), -2),
    (dict(t=dict(Wt=ODD)), -2), (dict(s=ODD), -2), (dict(add=ODD), -2), (dict(dX=ODD), -2),
    (dict(add=A, dX=None), -1), (dict(ws=None, M=300, t=dict(dbias=A)), -1),
    (dict(nbytes=8, M=300, t=dict(dbias=A)), -1), (dict(ws=A + 16, t=dict(dbias=A)), -2),
    (dict(count=2, terms=[term(), term(wbits=8)]), -3),
])
def test_linear_backward_refusals(kw, code):
    assert backward_rc(**kw) == code


def gated_backward_rc(g=None, u=None, dH=A, dX=A, M=1, K=128, dtype=0, ws=A, nbytes=1 << 30):
    g, u = term(**{"dY": None, **(g or {})}), term(**{"dY": None, "act": 0, **(u or {})})
    return w4.lib().w4a16_gated_backward(dH, ctypes.byref(g), ctypes.byref(u), None, None, dX, M, K, dtype,
                                         ws, nbytes, None)


@pytest.mark.parametrize("kw,code", [
    (dict(dH=None), -1), (dict(dH=ODD), -2), (dict(u=dict(N=32)), -1), (dict(u=dict(act=2)), -1),
    (dict(g=dict(preact=None)), -1), (dict(u=dict(preact=None)), -1), (dict(g=dict(dZ=None)), -1),
    (dict(u=dict(dZ=ODD)), -2), (dict(u=dict(wbits=8)), -3), (dict(g=dict(act=8)), -3), (dict(K=64), -1),
    (dict(dtype=-1), -3), (dict(g=dict(Wt=None)), -1), (dict(g=dict(dbias=A), M=300, ws=None), -1),
])
def test_gated_backward_refusals(kw, code):
    assert gated_backward_rc(**kw) == code


C, D, E = 1 << 22, 1 << 23, 1 << 24  # apart from A and B and each other


@pytest.mark.parametrize("kw", [
    dict(count=2, dX=E, terms=[term(dY=A, preact=B, dZ=A), term(dY=A, preact=C, dZ=D)]),   # dZ over a shared dY
    dict(count=2, dX=E, terms=[term(dY=A, preact=B, dZ=D), term(dY=C, preact=C, dZ=D)]),   # one dZ for both
    dict(count=2, dX=E, M=4, terms=[term(dY=A, preact=B, dZ=D), term(dY=C, preact=C, dZ=D + 64)]),
    dict(count=2, dX=E, terms=[term(dY=A, preact=B, dZ=C), term(dY=D, preact=C, dZ=D)]),   # another's preact
    dict(count=2, dX=E, terms=[term(dY=A, preact=B, dZ=C, dbias=1 << 25),
                               term(dY=D, preact=D, dZ=D, dbias=1 << 25)]),                # one dbias
    dict(dX=A, t=dict(dY=A, preact=B, dZ=C)), dict(dX=C, t=dict(dY=A, preact=B, dZ=C)),
    dict(dX=B, t=dict(dY=A, preact=B, dZ=C)), dict(dX=A, t=dict(dY=A, preact=None, dZ=None, act=0)),
])
def test_backward_refuses_outputs_over_what_is_still_read(kw):
    assert backward_rc(**kw) == -1


def test_gated_backward_refuses_outputs_over_what_is_still_read():
    G = dict(preact=B, dZ=B)
    assert gated_backward_rc(G, dict(preact=C, dZ=B), dH=D, dX=E) == -1
    assert gated_backward_rc(dict(preact=B, dZ=C), dict(preact=C, dZ=B), dH=D, dX=E) == -1
    assert gated_backward_rc(G, dict(preact=C, dZ=C), dH=D, dX=C) == -1


# Every buffer of a call of two terms in a megabyte of its own; M = 4, N = 128 and 256, K = 256.
AT = {n: (i + 8) << 20 for i, n in enumerate(
    ("dY0", "preact0", "dZ0", "dbias0", "Wt0", "meta0", "dY1", "preact1", "dZ1", "dbias1", "Wt1", "meta1",
     "s", "add", "dX", "ws"))}
OUTPUTS = ("dZ0", "dbias0", "dZ1", "dbias1", "dX")
IN_PLACE = {("dZ0", "dY0"), ("dZ0", "preact0"), ("dZ1", "dY1"), ("dZ1", "preact1"), ("dX", "add")}


def two_terms(at, M=4, act=2):
    n = {i: {f: at[f + str(i)] for f in ("dY", "preact", "dZ", "dbias", "Wt", "meta")} for i in (0, 1)}
    return backward_rc(count=2, terms=[term(N=128, act=act, **n[0]), term(N=256, act=act, **n[1])], s=at["s"],
                       add=at["add"], dX=at["dX"], M=M, K=256, ws=at["ws"])


@pytest.mark.parametrize("out", OUTPUTS)
@pytest.mark.parametrize("other", [n for n in AT if n != "ws"])
def test_backward_refuses_every_overlap(out, other):
    """An output at, inside or around another buffer of the call; only the named pairs may
    share an address (those run on the GPU)."""
    if out == other:
        return
    for offset in (0, 64, -64):
        if offset == 0 and (out, other) in IN_PLACE:
            continue
        assert two_terms({**AT, out: AT[other] + offset}) == -1, offset


def test_backward_refuses_a_dZ_into_a_dY_that_is_added():
    """The gradient of Y = X + act(X . W^T + b): add is dY, so dZ may not replace it."""
    assert backward_rc(dX=E, add=A, K=128, t=dict(dY=A, preact=B, dZ=A, N=128, Wt=C, meta=D)) == -1
    assert two_terms({**AT, "dZ0": AT["dY0"], "add": AT["dY0"]}) == -1
    assert two_terms({**AT, "dZ1": AT["preact1"], "add": AT["preact1"]}) == -1


def test_backward_of_no_rows_refuses_sums_over_inputs():
    """M = 0 still writes the bias gradients (zeros)."""
    for other in ("s", "Wt0", "meta1", "dbias1"):
        assert two_terms({**AT, "dbias0": AT[other]}, M=0) == -1


def test_gated_backward_refuses_every_overlap():
    at = {**AT, "dH": 64 << 20}

    def rc(at):
        g = term(dY=None, N=256, **{f: at[f + "0"] for f in ("preact", "dZ", "dbias", "Wt", "meta")})
        u = term(dY=None, N=256, act=0, **{f: at[f + "1"] for f in ("preact", "dZ", "dbias", "Wt", "meta")})
        return w4.lib().w4a16_gated_backward(at["dH"], ctypes.byref(g), ctypes.byref(u), at["s"], at["add"],
                                             at["dX"], 4, 256, 0, at["ws"], 1 << 20, None)
    for out in OUTPUTS:
        for other in at:
            if other in (out, "ws", "dY0", "dY1"):
                continue
            for offset in (0, 64, -64):
                if offset == 0 and ((out, other) in IN_PLACE or (out[:2], other) == ("dZ", "dH")):
                    continue
                assert rc({**at, out: at[other] + offset}) == -1, (out, other, offset)
    assert rc({**at, "dZ0": at["dH"], "add": at["dH"]}) == -1
    assert rc({**at, "dZ0": at["dH"], "dZ1": at["dH"]}) == -1


def test_backward_workspace_sizes():
    L, n = w4.lib(), ctypes.c_size_t()

    def size(t, M, K):
        assert L.w4a16_linear_backward_workspace_size(ctypes.byref(t), 1, M, K, 1, ctypes.byref(n)) == 0
        return n.value
    assert size(term(N=14336), 0, 4096) == 0
    assert size(term(N=128), 4096, 4096) == 0                       # nothing to split, no sums
    assert size(term(N=14336), 64, 256) > 0                         # few output blocks: N is split
    assert size(term(N=128, dbias=A), 4096, 4096) >= 4 * 128
    assert L.w4a16_linear_backward_workspace_size(ctypes.byref(term()), 1, 1, 128, 0, None) == -1
    g = term(N=16)
    assert L.w4a16_gated_backward_workspace_size(ctypes.byref(g), ctypes.byref(term(N=32)), 1, 128, 0,
                                                 ctypes.byref(n)) == -1


def test_binding_refusals():
    import torch
    x = torch.zeros(2, 128, dtype=torch.float16)                    # not a device tensor
    pw = w4.PackedWeight(None, None, None, 16, 128)
    with pytest.raises(TypeError):
        w4.LinearCall([(x, pw, None, x[:, :16].contiguous(), w4.Epilogue())])
    with pytest.raises(TypeError):
        w4.GatedCall(x.float(), pw, pw, None, x)
    with pytest.raises(ValueError):
        w4.GatedCall(x, pw, w4.PackedWeight(None, None, None, 32, 128), None, x)
    with pytest.raises(ValueError):
        w4.LinearBackwardCall([], None, None)
    w4.LinearCall([])()                                             # nothing to do


def test_binding_refuses_tensors_whose_gradient_would_be_lost():
    import torch
    x = torch.zeros(2, 128, dtype=torch.float16, requires_grad=True)
    y = torch.zeros(2, 16, dtype=torch.float16, requires_grad=True)
    pw, wt = w4.PackedWeight(None, None, None, 16, 128), w4.TransposedWeight(None, None, 16, 128)
    calls = (lambda: w4.LinearCall([(x, pw, None, y, w4.Epilogue())]),
             lambda: w4.GatedCall(x, pw, pw, None, y),
             lambda: w4.LinearBackwardCall([w4.BackwardTerm(y, wt)], None, x),
             lambda: w4.GatedBackwardCall(y, y, y, wt, wt, None, x, y, y))
    for call in calls:
        with pytest.raises(ValueError, match="requires grad"):
            call()
        with torch.no_grad(), pytest.raises(TypeError):              # not a device tensor
            call()


@pytest.mark.parametrize("source", ["backward.hip"])
def test_backward_kernels_keep_everything_in_registers(source, tmp_path):
    kernels = _kernel_metadata(_device_asm(source, tmp_path))
    assert kernels
    bad = [k for k in kernels if k[1] or k[2] or k[3]]
    assert not bad, f"{source}: (kernel, private bytes, VGPR spills, SGPR spills): {bad}"
