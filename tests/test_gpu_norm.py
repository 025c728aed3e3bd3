"""The norms before and after a block on the GPU, and their backward, against fp64.

Tolerances.  u is the activations' unit roundoff (eps / 2: 2^-11 fp16, 2^-8 bf16), e = 2^-24
that of fp32; TINY = 2^-25 is half the smallest fp16.  Errors are carried to first order:
  * a sum of D <= 16384 terms over a row runs as at most 32 terms a thread (one of 16, one FMA
    each, with its mean) and 10 additions of partial sums: 44 e relative to the sum of
    magnitudes.  The normalised row n = (v - mean) inv then carries
    N(v) = e * 64 * (|n| + mean|v| inv): 44 for each of the two sums (the second under a square
    root: half), the reciprocal root and three products.
  * an error e_v of the row moves n by inv (e_v + mean(e_v)) + |n| inv rms(e_v).
  * gradient of a norm, inv (d - m(d) - n m(d n)): with e_d on d and N on n,
    inv (e_d + m(e_d) + |n| m(e_d |n| + |d| N) + N |m(d n)|) + 64 e inv (|d| + m|d| + |n| m|d n|).
  * a sum over T rows: (T + 16) e times the sum of magnitudes, and the terms' errors.
Each output adds its own rounding, u times its value.
"""
import numpy as np
import pytest

import weight_only_int4_group_amd as w4
from oracle import block
from tests.gpu_helpers import note, torch_cuda

pytestmark = pytest.mark.gpu

E32, TINY = 2.0 ** -24, 2.0 ** -25
KIND = {"none": w4.NORM_NONE, "rms": w4.NORM_RMS, "layer": w4.NORM_LAYER}
EPS = 1e-5


def dtype_of(name):
    torch = torch_cuda()
    return {"fp16": torch.float16, "bf16": torch.bfloat16}[name]


def unit(name):
    return 2.0 ** -11 if name == "fp16" else 2.0 ** -8


class Data:
    """Seeded tensors of the activations' type and their fp64 values."""

    def __init__(self, dtype, *seed):
        self.torch, self.dt = torch_cuda(), dtype_of(dtype)
        self.rng = np.random.default_rng([17, *seed])

    def __call__(self, *shape, std=1.0, mean=0.0):
        x = (self.rng.standard_normal(shape) * std + mean).astype(np.float32)
        t = self.torch.from_numpy(x).to(self.dt).to("cuda")
        return t, t.double().cpu().numpy()


def values(t):
    torch_cuda().cuda.synchronize()
    return t.double().cpu().numpy()


def m(v):
    return v.mean(1, keepdims=True)


def norm_error(v, kind, weight, bias, eps, e_v):
    """Bound of the fp32 error of a norm's output whose input carries e_v."""
    if kind == "none":
        return e_v
    n, inv = block.normalized(v, kind, eps)
    own = 64 * E32 * (np.abs(n) + m(np.abs(v)) * inv)
    moved = inv * (e_v + m(e_v)) + np.abs(n) * inv * np.sqrt(m(e_v ** 2))
    w = 1.0 if weight is None else np.abs(weight)
    return w * (own + moved) + 4 * E32 * (w * np.abs(n) + (0.0 if bias is None else np.abs(bias)))


def check(got, ref, bound, tag):
    got = values(got)
    assert np.isfinite(got).all(), f"{tag}: non-finite"
    worst = (np.abs(got - ref) / bound).max()
    assert worst <= 1.0, f"{tag}: worst {worst:.3g} x bound"


def setup(T, D, dtype, post, pre, y, gate_rows, seed=0):
    a = Data(dtype, T, D, seed)
    t = {"x": a(T, D, std=2.0), "y": a(T, D, std=3.0, mean=0.5) if y else (None, None),
         "gate": a(-(-T // gate_rows), D, std=0.5) if gate_rows else (None, None)}
    for which, kind in (("post", post), ("pre", pre)):
        t[which + "_w"] = a(D, std=0.2, mean=1.0) if kind != "none" else (None, None)
        t[which + "_b"] = a(D, std=0.2) if kind == "layer" else (None, None)
    return a, t


def norms(t, post, pre):
    out = {}
    for which, kind in (("post", post), ("pre", pre)):
        dev = None if kind == "none" else w4.Norm(KIND[kind], t[which + "_w"][0], t[which + "_b"][0], EPS)
        out[which] = (dev, (kind, t[which + "_w"][1], t[which + "_b"][1], EPS))
    return out


def run_forward(T, D, dtype, post, pre, y=True, gate_rows=0, alpha=1.0, want_r=True, inplace=False):
    torch = torch_cuda()
    note(f"norm T={T} D={D} {dtype} post={post} pre={pre} y={y} gate={gate_rows} inplace={inplace}")
    _, t = setup(T, D, dtype, post, pre, y, gate_rows)
    n = norms(t, post, pre)
    u = unit(dtype)
    guard = [torch.full((T + 2, D), 777.0, dtype=dtype_of(dtype), device="cuda") for _ in range(2)]
    x, yt = t["x"][0], t["y"][0]
    r = x if inplace else guard[0][:T]
    h = yt if inplace and y else guard[1][:T]
    if pre == "none":
        h = None
    call = w4.NormBlockCall(x, yt, r if want_r else None, h, post=n["post"][0], pre=n["pre"][0],
                            gate=t["gate"][0], gate_rows=gate_rows or None, alpha=alpha)
    call()
    ref_r, ref_h = block.norm_block(t["x"][1], t["y"][1], n["post"][1], n["pre"][1], t["gate"][1],
                                    gate_rows or 1, alpha)
    e_r = 4 * E32 * np.abs(alpha * t["x"][1])
    if y:
        g = np.abs(block.gate_of(t["gate"][1], gate_rows, T))
        p = block.norm(t["y"][1], *n["post"][1])
        e_r = e_r + g * (norm_error(t["y"][1], *n["post"][1], np.zeros((T, D))) + 4 * E32 * np.abs(p))
    if want_r:
        check(r, ref_r, u * np.abs(ref_r) + 1.01 * e_r + TINY, "r")
    if h is not None:
        e_h = norm_error(ref_r, *n["pre"][1], e_r)
        check(h, ref_h, u * np.abs(ref_h) + 1.01 * e_h + TINY, "h")
    assert all(bool((b[T:] == 777.0).all()) for b in guard), "rows behind the output were written"


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("T,D", [(1, 4096), (3, 8), (5, 64), (2, 512), (7, 520), (4, 1024), (3, 2048), (2, 3584),
                                 (3, 8192), (2, 16384), (2, 16376)])
def test_widths(T, D, dtype):
    run_forward(T, D, dtype, "rms", "layer", gate_rows=2, alpha=0.5)


@pytest.mark.parametrize("T,D", [(3, 2), (9, 7), (5, 63), (2, 511), (3, 2049), (2, 4097), (2, 8191), (2, 16383)])
def test_odd_widths(T, D):
    run_forward(T, D, "bf16", "layer", "rms", gate_rows=2, alpha=1.5)


@pytest.mark.parametrize("post", block.KINDS)
@pytest.mark.parametrize("pre", block.KINDS)
@pytest.mark.parametrize("gate_rows", [0, 1, 3, 100])
def test_kinds(post, pre, gate_rows):
    run_forward(11, 136, "fp16", post, pre, gate_rows=gate_rows, alpha=-0.7)


def test_without_block_output_and_without_r():
    run_forward(6, 256, "bf16", "none", "rms", y=False)
    run_forward(6, 256, "bf16", "none", "rms", y=False, want_r=False)
    run_forward(6, 256, "bf16", "rms", "layer", want_r=False)
    run_forward(600, 72, "fp16", "rms", "rms")


@pytest.mark.parametrize("D", [96, 4096, 777])
def test_in_place(D):
    run_forward(5, D, "fp16", "rms", "rms", gate_rows=5, inplace=True)


def test_weights_default_to_one_and_zero_rows_are_finite():
    torch = torch_cuda()
    x = torch.randn(3, 640, device="cuda").half()
    x[1] = 0
    for kind in (w4.NORM_RMS, w4.NORM_LAYER):
        a = w4.w4a16_norm_block(x, pre=w4.Norm(kind, eps=1e-5))[1]
        b = w4.w4a16_norm_block(x, pre=w4.Norm(kind, torch.ones(640, device="cuda").half(),
                                               torch.zeros(640, device="cuda").half(), 1e-5))[1]
        assert torch.equal(a, b) and bool((a[1] == 0).all())


def test_large_mean_keeps_its_digits():
    """A layer norm of rows far from zero: the mean is taken before the squares."""
    torch = torch_cuda()
    x = (torch.arange(1024, device="cuda").half() % 8)[None] + 1000
    h = w4.w4a16_norm_block(x, pre=w4.Norm(w4.NORM_LAYER, eps=0.0))[1]
    v = x.double().cpu().numpy()
    ref = block.norm(v, "layer", eps=0.0)
    # N(v) with mean|v| inv = 1003.5 / 2.29
    check(h, ref, 2.0 ** -11 * np.abs(ref) + norm_error(v, "layer", None, None, 0.0, 0 * v), "h")


def test_nan_stays_in_its_row():
    torch = torch_cuda()
    x = torch.randn(4, 300, device="cuda").bfloat16()
    clean = w4.w4a16_norm_block(x, pre=w4.Norm(w4.NORM_LAYER))[1]
    x[2, 17] = float("nan")
    h = w4.w4a16_norm_block(x, pre=w4.Norm(w4.NORM_LAYER))[1]
    assert bool(torch.isnan(h[2]).all()) and torch.equal(h[[0, 1, 3]], clean[[0, 1, 3]])


def test_no_tokens():
    torch = torch_cuda()
    x = torch.empty(0, 64, dtype=torch.float16, device="cuda")
    r, h = w4.w4a16_norm_block(x, x, pre=w4.Norm())
    assert r.shape == h.shape == (0, 64)
    dx, dy, g = w4.w4a16_norm_block_backward(x, x, x, x, pre=w4.Norm(w4.NORM_RMS, torch.ones(64, device="cuda").half()))
    assert dx.shape == (0, 64) and bool((g.pre_weight == 0).all())


@pytest.mark.parametrize("rows", [None, 1, 0])
@pytest.mark.parametrize("how", ["current", "handle", "graph"])
def test_no_tokens_with_a_gate(rows, how):
    """A gate of one vector ([D] or [1][D]) or of none: its gradient is a sum over no rows, zeros, on the stream
    of the call."""
    torch = torch_cuda()
    D = 64
    note(f"norm without tokens, gate rows {rows}, {how}")
    x = torch.empty(0, D, dtype=torch.float16, device="cuda")
    gate = torch.ones(*([] if rows is None else [rows]), D, device="cuda").half()
    post, pre = (w4.Norm(w4.NORM_RMS, torch.ones(D, device="cuda").half()) for _ in range(2))
    r, h = w4.w4a16_norm_block(x, x, post=post, pre=pre, gate=gate)
    assert r.shape == h.shape == (0, D)
    sums = w4.NormGrads(torch.empty(gate.shape, device="cuda"), *(torch.empty(D, device="cuda") for _ in range(4)))
    sums.post_bias = sums.pre_bias = None
    side = torch.cuda.Stream()
    call = w4.NormBlockBackwardCall(x, x, x, x, torch.empty_like(x), torch.empty_like(x), sums, post, pre, gate,
                                    stream=side.cuda_stream if how == "handle" else None)
    got = [g for g in vars(sums).values() if g is not None]

    def fill():
        for g in got:
            g.fill_(float("nan"))
        torch.cuda.synchronize()
    fill()
    if how == "graph":
        side.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            call()
        for _ in range(3):
            fill()
            graph.replay()
            torch.cuda.synchronize()
            assert all(bool((g == 0).all()) for g in got)
    else:
        call()
        torch.cuda.synchronize()
        assert all(bool((g == 0).all()) for g in got)
    grads = w4.w4a16_norm_block_backward(x, x, x, x, post, pre, gate)[2]
    assert grads.gate.shape == gate.shape and bool((grads.gate == 0).all())


def test_nothing_to_do_returns_the_input():
    torch = torch_cuda()
    x = torch.randn(3, 40, device="cuda").half()
    r, h = w4.w4a16_norm_block(x)
    assert r is x and h is None
    r, h = w4.w4a16_norm_block(x, post=w4.Norm(w4.NORM_NONE))
    assert r is x and h is None
    with pytest.raises(ValueError):
        w4.w4a16_norm_block(x.t())


# ---- backward --------------------------------------------------------------------------------

def grad_error(d, v, kind, eps, e_d):
    """Bound of the fp32 error of a norm's input gradient, d (with e_d) being weight * dout."""
    n, inv = block.normalized(v, kind, eps)
    own_n = 64 * E32 * (np.abs(n) + m(np.abs(v)) * inv)
    mean = 1.0 if kind == "layer" else 0.0
    carried = e_d + mean * m(e_d) + np.abs(n) * m(e_d * np.abs(n) + np.abs(d) * own_n) + own_n * np.abs(m(d * n))
    return inv * carried + 64 * E32 * inv * (np.abs(d) + mean * m(np.abs(d)) + np.abs(n) * m(np.abs(d * n))), own_n


def run_backward(T, D, dtype, post, pre, y=True, gate_rows=0, alpha=1.0, with_dr=True, sums=True, seed=1):
    torch = torch_cuda()
    note(f"norm backward T={T} D={D} {dtype} post={post} pre={pre} y={y} gate={gate_rows} dr={with_dr} sums={sums}")
    a, t = setup(T, D, dtype, post, pre, y, gate_rows, seed)
    n = norms(t, post, pre)
    u = unit(dtype)
    dr = a(T, D, std=0.3) if with_dr else (None, None)
    dh = a(T, D, std=0.3) if pre != "none" else (None, None)
    r = a(T, D, std=2.0)
    f32 = lambda want, *shape: torch.full(shape, float("nan"), device="cuda") if want and sums else None  # noqa: E731
    grads = w4.NormGrads(f32(gate_rows, *(t["gate"][0].shape if gate_rows else ())), f32(post != "none", D),
                         f32(post == "layer", D), f32(pre != "none", D), f32(pre == "layer", D))
    dx, dy = torch.empty_like(r[0]), torch.empty_like(r[0]) if y else None
    call = w4.NormBlockBackwardCall(dr[0], dh[0], t["y"][0], r[0] if pre != "none" else None, dx, dy, grads,
                                    n["post"][0], n["pre"][0], t["gate"][0], gate_rows or None, alpha)
    call()
    first = [dx.clone()] + [None if g is None else g.clone() for g in vars(grads).values()]
    ref = block.norm_block_backward(dr[1], dh[1], t["y"][1], r[1], n["post"][1], n["pre"][1], t["gate"][1],
                                    gate_rows or 1, alpha)
    rows = T + 16
    # R and its error
    R = ref["dx"] / alpha
    e_R = np.zeros((T, D))
    if pre != "none":
        w = 1.0 if t["pre_w"][1] is None else t["pre_w"][1]
        d = dh[1] * w
        e, e_n = grad_error(d, r[1], pre, EPS, E32 * np.abs(d))
        nr = block.normalized(r[1], pre, EPS)[0]
        e_R = e + 2 * E32 * np.abs(R)
        if sums:
            mag = np.abs(dh[1] * nr)
            check(grads.pre_weight, ref["pre_weight"], (np.abs(dh[1]) * e_n).sum(0) + rows * E32 * mag.sum(0) + 1e-12,
                  "pre_weight")
            if pre == "layer":
                check(grads.pre_bias, ref["pre_bias"], rows * E32 * np.abs(dh[1]).sum(0) + 1e-12, "pre_bias")
    check(dx, ref["dx"], u * np.abs(ref["dx"]) + 1.01 * abs(alpha) * (e_R + 2 * E32 * np.abs(R)) + TINY, "dx")
    if y:
        g = block.gate_of(t["gate"][1], gate_rows, T)
        p = R * g
        e_p = np.abs(g) * e_R + E32 * np.abs(p)
        yv = t["y"][1]
        if gate_rows and sums:
            out = block.norm(yv, *n["post"][1])
            e = np.abs(R) * (norm_error(yv, *n["post"][1], np.zeros((T, D))) + 4 * E32 * np.abs(out)) + e_R * np.abs(out)
            per = lambda v: np.stack([v[b * gate_rows:(b + 1) * gate_rows].sum(0)  # noqa: E731
                                      for b in range(len(ref["gate"]))])
            check(grads.gate, ref["gate"], per(e) + rows * E32 * per(np.abs(R * out)) + 1e-12, "gate")
        if post == "none":
            check(dy, ref["dy"], u * np.abs(ref["dy"]) + 1.01 * e_p + TINY, "dy")
        else:
            w = 1.0 if t["post_w"][1] is None else t["post_w"][1]
            e, e_n = grad_error(p * w, yv, post, EPS, np.abs(w) * e_p + E32 * np.abs(p * w))
            check(dy, ref["dy"], u * np.abs(ref["dy"]) + 1.01 * e + TINY, "dy")
            if sums:
                ny = block.normalized(yv, post, EPS)[0]
                check(grads.post_weight, ref["post_weight"],
                      (np.abs(p) * e_n + e_p * np.abs(ny)).sum(0) + rows * E32 * np.abs(p * ny).sum(0) + 1e-12,
                      "post_weight")
                if post == "layer":
                    check(grads.post_bias, ref["post_bias"], e_p.sum(0) + rows * E32 * np.abs(p).sum(0) + 1e-12,
                          "post_bias")
    call()  # the same bits again
    torch.cuda.synchronize()
    for x, g in zip(first, [dx] + list(vars(grads).values())):
        assert x is None or torch.equal(x, g)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("T,D", [(1, 64), (3, 8), (33, 512), (17, 1024), (20, 2048), (9, 4096), (10, 8192),
                                 (11, 8200), (9, 16384)])
def test_backward_widths(T, D, dtype):
    run_backward(T, D, dtype, "rms", "layer", gate_rows=4, alpha=0.5)


@pytest.mark.parametrize("T,D", [(5, 7), (19, 63), (9, 513), (10, 4099), (9, 16383)])
def test_backward_odd_widths(T, D):
    run_backward(T, D, "bf16", "layer", "rms", gate_rows=4, alpha=2.0)


@pytest.mark.parametrize("post", block.KINDS)
@pytest.mark.parametrize("pre", block.KINDS)
@pytest.mark.parametrize("gate_rows", [0, 1, 5, 64, 1000])
def test_backward_kinds(post, pre, gate_rows):
    """Gates within a strip of rows, and strips within a gate."""
    run_backward(203, 72, "bf16", post, pre, gate_rows=gate_rows, alpha=0.7)


@pytest.mark.parametrize("D", [256, 10000, 77])
def test_backward_parts(D):
    run_backward(21, D, "fp16", "none", "rms", y=False)
    run_backward(21, D, "fp16", "rms", "layer", with_dr=False)
    run_backward(21, D, "fp16", "layer", "rms", sums=False)


def test_backward_many_rows():
    """Strips of more than eight rows, several a gate, the last gate's rows cut short."""
    run_backward(40001, 16, "fp16", "rms", "rms", gate_rows=9000)
    run_backward(20000, 24, "bf16", "layer", "none", gate_rows=3)


@pytest.mark.parametrize("post", block.KINDS)
@pytest.mark.parametrize("gate_rows", [64, 1000])
@pytest.mark.parametrize("D", [77, 8200])
def test_backward_long_gates_of_rows_in_two_passes(D, gate_rows, post):
    """Widths whose sums have a kernel of their own, gates of several strips of rows, the last one cut short."""
    run_backward(203, D, "fp16" if D == 77 else "bf16", post, "rms", gate_rows=gate_rows, alpha=0.7)


def test_backward_many_rows_in_two_passes():
    """As above with strips of more than eight rows; and strips of several gates, the last one cut short."""
    run_backward(40001, 17, "fp16", "rms", "layer", gate_rows=9000)
    run_backward(40001, 13, "bf16", "layer", "none", gate_rows=3)
    run_backward(4200, 8200, "bf16", "rms", "none", gate_rows=1000)


def test_backward_against_differences():
    """dx and dy of a few elements against differences of the forward's fp64 values through the
    library's own rows (an fp16 step of 1/16 about a smooth point)."""
    torch = torch_cuda()
    rng = np.random.default_rng(3)
    x = torch.from_numpy(rng.standard_normal((1, 32)).astype(np.float32)).half().cuda()
    y = torch.from_numpy(rng.standard_normal((1, 32)).astype(np.float32)).half().cuda()
    post, pre = w4.Norm(w4.NORM_RMS, eps=1e-2), w4.Norm(w4.NORM_LAYER, eps=1e-2)
    r, h = w4.w4a16_norm_block(x, y, post, pre)
    d = torch.ones_like(h) * torch.linspace(-1, 1, 32, device="cuda").half()
    dx, dy, _ = w4.w4a16_norm_block_backward(None, d, y, r, post, pre)

    def f(x, y):
        _, h = w4.w4a16_norm_block(x, y, post, pre)
        return float((h.double() * d.double()).sum())
    step = 2.0 ** -4
    for grad, t, call in ((dx, x, lambda v: f(v, y)), (dy, y, lambda v: f(x, v))):
        for i in (0, 9, 31):
            a, b = t.double(), t.double()
            a[0, i] += step
            b[0, i] -= step
            ah, bh = a.half(), b.half()
            est = (call(ah) - call(bh)) / float(ah[0, i].double() - bh[0, i].double())
            # 32 outputs below 2.5 rounded to fp16 on each side: 2 * 32 * 2.5 * 2^-11 * rms(d) 0.58 over
            # 2 * step, as independent errors over sqrt(64); the third derivative's step^2 / 6 below 0.01
            assert abs(est - float(grad[0, i])) <= 0.05 + 0.01


def test_graph_streams_and_shared_workspace():
    torch = torch_cuda()
    T, D = 300, 512
    a, t = setup(T, D, "bf16", "rms", "layer", True, 100)
    n = norms(t, "rms", "layer")
    dr, dh, r = a(T, D)[0], a(T, D)[0], a(T, D)[0]
    h, rr, dx, dy = (torch.empty(T, D, dtype=torch.bfloat16, device="cuda") for _ in range(4))
    grads = w4.NormGrads(torch.empty(3, D, device="cuda"), *(torch.empty(D, device="cuda") for _ in range(4)))
    grads.post_bias = None
    fwd = w4.NormBlockCall(t["x"][0], t["y"][0], rr, h, n["post"][0], n["pre"][0], t["gate"][0], 100)
    bwd = w4.NormBlockBackwardCall(dr, dh, t["y"][0], r, dx, dy, grads, n["post"][0], n["pre"][0], t["gate"][0], 100)
    outs = [rr, h, dx, dy] + [g for g in vars(grads).values() if g is not None]

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
        t["y"][0].mul_(1.1)
        dh.add_(0.1)
        want = expect()
        for o in outs:
            o.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want)), f"replay {i}"
    side = torch.cuda.Stream()
    want = expect()
    for o in outs:
        o.fill_(float("nan"))
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        fwd()
        bwd()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_past_32_bit_offsets():
    """Rows whose offsets pass 2^32 bytes, at the end of the largest batch of this width."""
    torch = torch_cuda()
    D, T = 4096, 540000      # 4.4 GB a tensor
    x = torch.zeros(T, D, dtype=torch.float16, device="cuda")
    g = torch.Generator("cuda").manual_seed(1)
    x[-5:] = torch.randn(5, D, device="cuda", generator=g).half()
    h = torch.empty_like(x)
    n = w4.Norm(w4.NORM_RMS)
    note("norm past 32 bits")
    w4.NormBlockCall(x, None, None, h, pre=n)()
    small = w4.w4a16_norm_block(x[-8:].clone(), pre=n)[1]
    assert torch.equal(h[-8:], small) and bool((h[:-5:1000] == 0).all())
    dx = torch.empty_like(x)
    w4.NormBlockBackwardCall(None, h, None, x, dx, None, pre=n)()
    one = torch.empty_like(x[-8:])
    w4.NormBlockBackwardCall(None, h[-8:].clone(), None, x[-8:].clone(), one, None, pre=n)()
    assert torch.equal(dx[-8:], one)
