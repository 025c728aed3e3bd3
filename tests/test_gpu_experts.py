"""The experts' products on the GPU, and their backward, against the fp64 oracle.

Tolerances.  u is the activations' unit roundoff (2^-11 fp16, 2^-8 bf16), e = 2^-24 fp32's, TINY = 2^-25 half
the smallest fp16.  Errors are carried to first order, with a factor 1.05 for the rest.
  * A forward product multiplies exact codes: per group of 128 the MFMA's fp32 sum of x (c + q), c = 64 (fp16) or
    128 (bf16), and that of x, at most 40 additions deep each, then two FMAs per group.  Its error is
    (40 + groups + 4) e times B = sum |x| scale 2 (c + 16); X * s adds u times sum |x s| |w|.
  * With more than 56 slots per expert a product may round each weight (u, or TINY where it is below fp16's
    normal numbers) and sum in fp32 instead, K additions deep: (u + (K + 8) e) sum |x| |w| + TINY sum |x|.
  * act: slopes within 1.2, fp32 evaluation within 2^-19 (1 + |z|); H = act(G) U s_down, rounded (u).
  * The token's sum: (k + 2) e of the magnitudes; Y is rounded (u).
  * A backward product rounds each weight (u) and sums in fp32: (u + (R + 8) e) times sum |x| |w|.
"""
import numpy as np
import pytest

import oracle
import weight_only_int4_group_amd as w4
from oracle import block
from oracle import fused as of
from tests.gpu_helpers import note, to_dev, to_host, torch_cuda
from workloads import weights

pytestmark = pytest.mark.gpu

E32, TINY = 2.0 ** -24, 2.0 ** -25
ACT = {n: getattr(w4, "ACT_" + n.upper()) for n in of.ACTS}
_STACKS = {}


def unit(dtype):
    return 2.0 ** -11 if dtype == "fp16" else 2.0 ** -8


class Stack:
    """E packed weights [N][K]: the library's, their fp64 values and their scales per column."""

    def __init__(self, key, E, N, K):
        torch_cuda()
        packed = [w4.w4a16_quantize_pack(to_dev(weights(61, 100 * key + e, N, K))) for e in range(E)]
        self.dev = w4.w4a16_stack_experts(packed)
        self.scale = np.stack([np.repeat(oracle.unpack_meta(to_host(p.scales), N, K).astype(np.float64), 128, 1)
                               for p in packed])
        self.W = np.stack([oracle.dequantize(oracle.unpack_codes(to_host(p.wq), N, K),
                                             oracle.unpack_meta(to_host(p.scales), N, K),
                                             oracle.unpack_meta(to_host(p.zeros), N, K)) for p in packed])
        self.T = None

    def transposed(self):
        if self.T is None:
            self.T = w4.w4a16_transpose_experts(self.dev)
        return self.T


def stack(key, E, N, K):
    k = (key, E, N, K)
    if k not in _STACKS:
        if len(_STACKS) > 40:
            _STACKS.clear()
        _STACKS[k] = Stack(*k)
    return _STACKS[k]


def tensor(dtype, seed, *shape, std=1.0):
    torch = torch_cuda()
    x = (np.random.default_rng([71, seed, *shape]).standard_normal(shape) * std).astype(np.float32)
    t = torch.from_numpy(x).to(torch.float16 if dtype == "fp16" else torch.bfloat16).cuda()
    return t, t.double().cpu().numpy()


def routing(T, E, k, kind="even", seed=0):
    rng = np.random.default_rng([73, T, E, k, seed])
    if kind == "same":                    # all tokens the same experts
        ids = np.tile(np.arange(E - k, E), (T, 1))
    elif kind == "double":                # the same expert in every slot of a token
        ids = np.repeat(rng.integers(0, E, (T, 1)), k, 1)
    else:
        ids = np.argsort(rng.random((T, E)), 1)[:, :k]
    if kind == "skip":                    # padded tokens and experts held elsewhere
        ids = np.where(rng.random((T, k)) < 0.4, rng.choice([-1, E, E + 7, -(1 << 30)], (T, k)), ids)
    if kind == "none":
        ids = np.full((T, k), -1)
    w = (rng.random((T, k)) + 0.1).astype(np.float32)
    return ids.astype(np.int32), w


def product(x, W, scale, e_x, dtype, rounded=False):
    """(x . W^T, its fp32 error with e_x on x; rounded: or that of rounded weights)."""
    c = 64 if dtype == "fp16" else 128
    K = x.shape[1]
    B = np.abs(x) @ (scale * 2 * (c + 16)).T
    own = (44 + K // 128) * E32 * B
    if rounded:
        own = np.maximum(own, (unit(dtype) + (K + 8) * E32) * (np.abs(x) @ np.abs(W).T) +
                         TINY * np.abs(x).sum(1, keepdims=True))
    return x @ W.T, own + e_x @ np.abs(W).T


def forward_bounds(Xv, ids, w, st, dtype, act, s, s_down, residual, rounded=None):
    """The oracle's (Y, G, U) and bounds of each."""
    gate, up, down = st
    u = unit(dtype)
    Y, G, U = block.experts(Xv, ids, w.astype(np.float64), gate.W, up.W, down.W, act, s, s_down, residual)
    bY, bG, bU = np.zeros_like(Y), np.zeros_like(G), np.zeros_like(U)
    mag = np.zeros_like(Y) if residual is None else np.abs(residual)
    if rounded is None:
        rounded = ids.size > 56 * min(gate.W.shape[0], ids.size)
    xs = Xv if s is None else Xv * s
    e_x = np.zeros_like(xs) if s is None else u * np.abs(xs) + TINY
    for e in range(gate.W.shape[0]):
        t, j = np.nonzero(ids == e)
        if not len(t):
            continue
        g, eg = product(xs[t], gate.W[e], gate.scale[e], e_x[t], dtype, rounded)
        uu, eu = product(xs[t], up.W[e], up.scale[e], e_x[t], dtype, rounded)
        sd = 1.0 if s_down is None else s_down[e]
        a = of.act(g, act)
        ea = 1.2 * eg + 2.0 ** -19 * (1 + np.abs(g))
        h = a * uu * sd
        eh = sd * (ea * (np.abs(uu) + eu) + np.abs(a) * eu) + (u + 4 * E32) * np.abs(h) + TINY
        p, ep = product(h, down.W[e], down.scale[e], eh, dtype, rounded)
        bG[t, j], bU[t, j] = 1.05 * eg + u * np.abs(g) + TINY, 1.05 * eu + u * np.abs(uu) + TINY
        wt = w[t, j][:, None].astype(np.float64)
        np.add.at(bY, t, wt * ep)
        np.add.at(mag, t, wt * np.abs(p))
    bY = 1.05 * (bY + (ids.shape[1] + 4) * E32 * mag) + u * np.abs(Y) + TINY
    return (Y, G, U), (bY, bG, bU)


def check(got, ref, bound, tag):
    torch_cuda().cuda.synchronize()
    v = got.double().cpu().numpy()
    assert np.isfinite(v).all(), f"{tag}: non-finite"
    worst = (np.abs(v - ref) / bound).max(initial=0.0)
    assert worst <= 1.0, f"{tag}: worst {worst:.3g} x bound"


def scales(E, D, N, on):
    if not on:
        return None, None, None, None
    rng = np.random.default_rng([79, E, D, N])
    s, sd = np.exp(0.5 * rng.standard_normal(D)).astype(np.float16), np.exp(0.5 * rng.standard_normal((E, N))).astype(np.float16)
    return to_dev(s), to_dev(sd), s.astype(np.float64), sd.astype(np.float64)


def run_forward(T, E, k, D, N, dtype="bf16", act="silu", kind="even", s=False, residual=False, train=False, inplace=False):
    torch = torch_cuda()
    note(f"experts T={T} E={E} k={k} D={D} N={N} {dtype} {act} {kind} s={s} residual={residual} train={train}")
    st = stack(1, E, N, D), stack(2, E, N, D), stack(3, E, D, N)
    X, Xv = tensor(dtype, 1, T, D)
    R, Rv = tensor(dtype, 2, T, D) if residual else (None, None)
    ids, w = routing(T, E, k, kind)
    sd, sdd, sv, sdv = scales(E, D, N, s)
    dt = X.dtype
    Ybuf = torch.full((T + 2, D), 777.0, dtype=dt, device="cuda")
    Y = Ybuf[:T]
    if inplace:
        Y.copy_(R)
        R = Y
    pre = tuple(torch.full((T, k, N), 555.0, dtype=dt, device="cuda") for _ in range(2)) if train else None
    call = w4.ExpertsCall(X, to_dev(ids), to_dev(w), *(x.dev for x in st), Y, s=sd, s_down=sdd, act=ACT[act], residual=R,
                          preact=pre)
    call.ws.fill_(0x7f)                       # whatever a workspace held before
    call()
    refs, bounds = forward_bounds(Xv, ids, w, st, dtype, act, sv, sdv, Rv)
    check(Y, refs[0], bounds[0], "Y")
    assert bool((Ybuf[T:] == 777.0).all()), "rows behind the output were written"
    if train:
        on = (ids >= 0) & (ids < E)
        for p, ref, b, tag in zip(pre, refs[1:], bounds[1:], "GU"):
            assert bool((p[to_dev(~on)] == 555.0).all()), f"{tag}: a skipped slot was written"
            check(p[to_dev(on)], ref[on], b[on], tag)
    if not inplace:
        first = Y.clone()
        call()
        assert torch.equal(Y, first), "the same call gave other bits"
    return X, ids, w, st


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("T,E,k,D,N", [(1, 1, 1, 128, 128), (1, 4, 2, 256, 384), (3, 8, 3, 640, 128), (16, 4, 2, 384, 640),
                                       (33, 2, 1, 256, 256), (40, 3, 2, 128, 384), (70, 2, 2, 512, 128),
                                       (200, 3, 2, 384, 256), (130, 1, 1, 256, 640), (64, 16, 8, 256, 128),
                                       # tiles of 16, 32, 64 and 128 rows
                                       (56, 512, 8, 128, 128), (448, 512, 8, 128, 128), (2000, 512, 8, 128, 128),
                                       (2900, 512, 32, 128, 128), (200, 40, 8, 256, 1024), (5500, 4, 4, 640, 384),
                                       # and the contraction in two parts and in four
                                       (1900, 2, 2, 128, 2176), (60, 2, 1, 128, 8192)])
def test_shapes(T, E, k, D, N, dtype):
    run_forward(T, E, k, D, N, dtype)


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("T", [2, 100])
def test_activations(T, act):
    run_forward(T, 4, 2, 256, 256, "bf16", act, s=True, train=True)


@pytest.mark.parametrize("kind", ["same", "double", "skip", "none"])
@pytest.mark.parametrize("T", [1, 7, 60, 300])
def test_routings(T, kind):
    run_forward(T, 5, 2, 256, 128, "fp16", kind=kind, residual=T > 7, train=True)


def test_rounded_weights_with_scales_and_kept_products():
    for dtype in ("fp16", "bf16"):
        run_forward(1800, 2, 2, 256, 2176, dtype, "gelu", s=True, residual=True, train=True)
        run_forward(2600, 3, 2, 128, 2048, dtype, kind="skip", residual=True, train=True)


def test_residual_in_place():
    run_forward(9, 4, 2, 256, 256, "bf16", residual=True, inplace=True)
    run_forward(150, 4, 2, 256, 256, "fp16", s=True, residual=True, inplace=True)


def test_long_contraction_and_many_experts():
    run_forward(5, 3, 2, 4096, 128, "bf16")
    run_forward(5, 3, 2, 128, 4096, "fp16")
    run_forward(90, 2, 1, 128, 2048, "bf16")
    run_forward(50, 130, 8, 128, 128, "fp16", kind="skip")


@pytest.mark.parametrize("T,E,k,D,N", [(5, 4, 2, 256, 128), (40, 3, 2, 256, 384), (200, 40, 8, 256, 1024),
                                       (1900, 2, 2, 128, 2176)])
def test_nothing_of_padded_tokens_is_read(T, E, k, D, N):
    """Tokens without an expert hold NaN, their weights and kept products too; the others give the bits that they
    give beside finite ones, and a padded token's row is the residual."""
    torch = torch_cuda()
    note(f"experts padded T={T} E={E} k={k} D={D} N={N}")
    st = stack(1, E, N, D), stack(2, E, N, D), stack(3, E, D, N)
    ids, w = routing(T, E, k)
    pad = np.arange(T) % 3 == 1
    ids[pad] = -1
    X, _ = tensor("bf16", 41, T, D)
    R, _ = tensor("bf16", 42, T, D)
    dY, _ = tensor("bf16", 43, T, D)
    idd, wd, off = to_dev(ids), to_dev(w), to_dev(pad)
    G, U = (torch.zeros(T, k, N, dtype=X.dtype, device="cuda") for _ in range(2))
    back = [x.transposed() for x in st]

    def run():
        Y = w4.w4a16_experts(X, idd, wd, *(x.dev for x in st), residual=R, preact=(G, U))
        return (Y, *w4.w4a16_experts_backward(dY, idd, wd, G, U, *back, add=R))
    want = [t.clone() for t in run()]
    for t in (X, dY, G, U, wd):
        t[off] = float("nan")
    got = run()
    assert all(bool(torch.isfinite(t).all()) for t in got)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert torch.equal(got[0][off], R[off]) and torch.equal(got[1][off], R[off]) and bool((got[2][off] == 0).all())


def test_most_experts_and_slots():
    run_forward(3, 1024, 64, 128, 128, "bf16", s=True, train=True)
    run_backward(3, 1024, 64, 128, 128, "fp16", f32=True)


def test_no_tokens():
    torch = torch_cuda()
    st = stack(1, 2, 128, 128), stack(2, 2, 128, 128), stack(3, 2, 128, 128)
    X = torch.empty(0, 128, dtype=torch.float16, device="cuda")
    ids, w = torch.empty(0, 2, dtype=torch.int32, device="cuda"), torch.empty(0, 2, device="cuda")
    assert w4.w4a16_experts(X, ids, w, *(x.dev for x in st)).shape == (0, 128)
    G = torch.empty(0, 2, 128, dtype=torch.float16, device="cuda")
    dX, dw = w4.w4a16_experts_backward(X, ids, w, G, G, *(x.transposed() for x in st))
    assert dX.shape == (0, 128) and dw.shape == (0, 2)


def test_more_slots_than_a_round_holds():
    """2 x 70000 slots run in two rounds, of 65536 and 4464 tokens."""
    torch = torch_cuda()
    st = stack(1, 4, 128, 128), stack(2, 4, 128, 128), stack(3, 4, 128, 128)
    X, Xv = tensor("bf16", 5, 70000, 128)
    ids, w = routing(70000, 4, 2, "skip")
    on = (ids >= 0) & (ids < 4)
    idd, wd = to_dev(ids), to_dev(w)
    pre = tuple(torch.zeros(70000, 2, 128, dtype=X.dtype, device="cuda") for _ in range(2))
    note("experts in rounds")
    Y = w4.w4a16_experts(X, idd, wd, *(x.dev for x in st), residual=X, preact=pre)
    dY, _ = tensor("bf16", 6, 70000, 128)
    back = [x.transposed() for x in st]
    dX, dw = w4.w4a16_experts_backward(dY, idd, wd, *pre, *back, add=dY)
    for a in (0, 65000, 69000):
        r = slice(a, a + 1000)
        refs, bounds = forward_bounds(Xv[r], ids[r], w[r], st, "bf16", "silu", None, None, Xv[r], rounded=True)
        check(Y[r], refs[0], bounds[0], "Y")
        for p, ref, b, tag in zip(pre, refs[1:], bounds[1:], "GU"):
            assert bool((p[r][to_dev(~on[r])] == 0).all()), f"{tag}: a skipped slot was written"
            check(p[r][to_dev(on[r])], ref[on[r]], b[on[r]], tag)
        # (two stages of contraction: never split, and of one order in every tile)
        dx, d = w4.w4a16_experts_backward(dY[r], idd[r], wd[r], *(p[r] for p in pre), *back, add=dY[r])
        assert torch.equal(dX[r], dx) and torch.equal(dw[r], d)


def test_weights_past_32_bit_offsets():
    """The last of 80 experts, 4.7 GB into each weight, gives the bits of the same expert as the last of two
    (two tiles at most in both calls, so the contraction is split alike)."""
    torch = torch_cuda()
    E, D, N = 80, 4096, 28672
    g = torch.Generator("cuda").manual_seed(4)

    def packed(n, c):
        codes = torch.randint(0, 256, (E * n * c // 2,), dtype=torch.uint8, device="cuda", generator=g)
        meta = n * ((c // 128 + 3) // 4 * 4)
        sc = torch.rand(E * meta, device="cuda", generator=g).half() * 0.01
        return w4.PackedExperts(codes, sc, torch.full((E * meta,), 8.0, dtype=torch.float16, device="cuda"), E, n, c)

    def last(w):
        part = [v.view(E, -1)[E - 2:].reshape(-1).clone() for v in (w.wq, w.scales, w.zeros)]
        return w4.PackedExperts(*part, 2, w.N, w.K)
    three = [packed(N, D), packed(N, D), packed(D, N)]
    X, _ = tensor("fp16", 7, 2, D)
    w = torch.ones(2, 1, device="cuda")
    note("experts past 32 bits")
    Y = w4.w4a16_experts(X, torch.full((2, 1), E - 1, dtype=torch.int32, device="cuda"), w, *three)
    two = w4.w4a16_experts(X, torch.ones(2, 1, dtype=torch.int32, device="cuda"), w, *(last(x) for x in three))
    assert torch.equal(Y, two) and bool(torch.isfinite(Y).all()) and bool((Y != 0).any())


# ---- backward --------------------------------------------------------------------------------

def run_backward(T, E, k, D, N, dtype="bf16", act="silu", kind="even", s=False, add=False, want_dx=True, want_dw=True,
                 f32=False):
    torch = torch_cuda()
    note(f"experts backward T={T} E={E} k={k} D={D} N={N} {dtype} {act} {kind} s={s} add={add}")
    st = stack(1, E, N, D), stack(2, E, N, D), stack(3, E, D, N)
    dY, dYv = tensor(dtype, 11, T, D)
    G, Gv = tensor(dtype, 12, T, k, N)
    U, Uv = tensor(dtype, 13, T, k, N)
    A, Av = tensor(dtype, 14, T, D) if add else (None, None)
    ids, w = routing(T, E, k, kind)
    sd, sdd, sv, sdv = scales(E, D, N, s)
    off = to_dev((ids < 0) | (ids >= E))
    G[off], U[off] = float("nan"), float("inf")       # a skipped slot's are not read
    buf = torch.full((T + 2, D), 777.0, dtype=dY.dtype, device="cuda")
    dX = buf[:T] if want_dx else None
    dw = torch.full((T, k), float("nan"), dtype=torch.float32 if f32 else dY.dtype, device="cuda") if want_dw else None
    call = w4.ExpertsBackwardCall(dY, to_dev(ids), to_dev(w), G, U, *(x.transposed() for x in st), dX, dw, s=sd, s_down=sdd,
                                  act=ACT[act], add=A)
    call.ws.fill_(0x7f)
    call()
    gate, up, down = (x.W for x in st)
    rX, rw = block.experts_backward(dYv, ids, w.astype(np.float64), Gv, Uv, gate, up, down, act, sv, sdv, Av)
    u = unit(dtype)
    bX, bw, mag = np.zeros((T, D)), np.zeros((T, k)), np.zeros((T, D))
    for e in range(E):
        t, j = np.nonzero(ids == e)
        if not len(t):
            continue
        g, uu, wt = Gv[t, j], Uv[t, j], w[t, j][:, None].astype(np.float64)
        q = 1.0 if sdv is None else sdv[e]
        dh = q * (dYv[t] @ down[e])
        e_dh = q * (u + (D + 8) * E32) * (np.abs(dYv[t]) @ np.abs(down[e])) + q * TINY * np.abs(dYv[t]).sum(1, keepdims=True)
        a, da = of.act(g, act), of.act_grad(g, act)
        ea = 2.0 ** -19 * (1 + np.abs(g)) * (1 + np.abs(g))
        bw[t, j] = (e_dh * np.abs(a * uu) + np.abs(dh * uu) * ea).sum(1) + (N + 80) * E32 * np.abs(dh * a * uu).sum(1)
        dG, dU = wt * dh * uu * da, wt * dh * a
        e_dG = wt * np.abs(uu) * (e_dh * np.abs(da) + np.abs(dh) * ea) + (u + 4 * E32) * np.abs(dG) + TINY
        e_dU = wt * (e_dh * np.abs(a) + np.abs(dh) * ea) + (u + 4 * E32) * np.abs(dU) + TINY
        aW, bW = np.abs(gate[e]), np.abs(up[e])
        own = u + (2 * N + 8) * E32
        np.add.at(bX, t, e_dG @ aW + e_dU @ bW + own * (np.abs(dG) @ aW + np.abs(dU) @ bW) +
                  TINY * (np.abs(dG) + np.abs(dU)).sum(1, keepdims=True))
        np.add.at(mag, t, np.abs(dG) @ aW + np.abs(dU) @ bW)
    sq = 1.0 if sv is None else sv
    if want_dx:
        extra = 0.0 if Av is None else E32 * np.abs(Av)
        check(dX, rX, 1.05 * sq * (bX + (k + 4) * E32 * mag) + extra + u * np.abs(rX) + TINY, "dX")
        assert bool((buf[T:] == 777.0).all()), "rows behind the output were written"
    if want_dw:
        check(dw, rw, 1.05 * bw + (E32 if f32 else u) * np.abs(rw) + TINY, "dweights")
    first = [None if x is None else x.clone() for x in (dX, dw)]
    call()
    for x, y in zip(first, (dX, dw)):
        assert x is None or torch.equal(x, y), "the same call gave other bits"


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("T,E,k,D,N", [(1, 1, 1, 128, 128), (1, 4, 2, 256, 384), (16, 4, 2, 384, 640), (40, 3, 2, 128, 384),
                                       (70, 2, 2, 512, 128), (90, 3, 2, 384, 256), (300, 2, 1, 256, 640),
                                       (64, 16, 8, 256, 128), (32, 2, 2, 128, 256), (330, 2, 1, 256, 128),
                                       (200, 1, 1, 128, 384),
                                       # tiles of 16, 32, 64 and 128 rows
                                       (448, 512, 8, 128, 128), (960, 512, 8, 128, 128), (448, 512, 32, 128, 128),
                                       (928, 512, 32, 128, 128),
                                       # and the contraction in two parts and in four
                                       (90, 3, 2, 384, 768), (8, 3, 2, 128, 4096), (1900, 2, 2, 256, 4352)])
def test_backward_shapes(T, E, k, D, N, dtype):
    run_backward(T, E, k, D, N, dtype)


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "gelu_tanh"])
def test_backward_activations(act):
    run_backward(30, 4, 2, 256, 256, "bf16", act, s=True, add=True)


@pytest.mark.parametrize("kind", ["same", "double", "skip", "none"])
@pytest.mark.parametrize("T", [1, 60, 300])
def test_backward_routings(T, kind):
    run_backward(T, 5, 2, 256, 128, "fp16", kind=kind, add=T > 1)


def test_backward_parts():
    run_backward(20, 4, 2, 128, 256, want_dx=False)
    run_backward(20, 4, 2, 128, 256, want_dw=False, s=True)
    run_backward(20, 4, 2, 128, 256, want_dx=False, f32=True)
    run_backward(70, 3, 2, 256, 384, "fp16", kind="skip", s=True, add=True, f32=True)


def test_graphs_streams_and_workspaces():
    torch = torch_cuda()
    for T in (3, 90):
        E, k, D, N = 4, 2, 256, 256
        st = stack(1, E, N, D), stack(2, E, N, D), stack(3, E, D, N)
        X, _ = tensor("bf16", 21, T, D)
        ids, w = (to_dev(x) for x in routing(T, E, k))
        G, U = (torch.empty(T, k, N, dtype=X.dtype, device="cuda") for _ in range(2))
        Y, dX = torch.empty_like(X), torch.empty_like(X)
        dw = torch.empty(T, k, dtype=X.dtype, device="cuda")
        fwd = w4.ExpertsCall(X, ids, w, *(x.dev for x in st), Y, preact=(G, U))
        bwd = w4.ExpertsBackwardCall(Y, ids, w, G, U, *(x.transposed() for x in st), dX, dw)
        outs = (Y, G, U, dX, dw)

        def expect():
            fwd()
            bwd()
            torch.cuda.synchronize()
            return [o.clone() for o in outs]
        expect()
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            fwd()
            bwd()
        for i in range(4):
            X.mul_(0.9)
            ids.copy_((ids + 1) % E)              # another plan on every replay
            want = expect()
            for o in outs:
                o.zero_()
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(outs, want)), f"T={T} replay {i}"
        # another stream, and a caller's larger workspace
        want = expect()
        ws = torch.empty(fwd.ws_bytes + 4096, dtype=torch.uint8, device="cuda")
        other = torch.empty_like(Y)
        call = w4.ExpertsCall(X, ids, w, *(x.dev for x in st), other, workspace=ws)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            call()
        side.synchronize()
        assert torch.equal(other, want[0])


@pytest.mark.parametrize("T,E,k,kind", [(50, 130, 8, "skip"), (448, 512, 8, "even"), (3, 1024, 64, "even")])
def test_every_expert_has_weights_of_its_own(monkeypatch, T, E, k, kind):
    """Stacks whose seeds lie further apart than there are experts: no expert of one has the weights of another
    expert of another stack."""
    plain = stack
    monkeypatch.setitem(globals(), "stack", lambda key, *shape: plain(20 * key, *shape))
    run_forward(T, E, k, 128, 128, "fp16", kind=kind, s=True, train=True)
    run_backward(T, E, k, 128, 128, "bf16", kind=kind, f32=True)
