"""Routing of tokens to experts on the GPU, and its backward, against the fp64 oracle.

Choices have to be equal.  Weights come from 64-bit arithmetic and are rounded to fp32 once:
2^-24 of their value, and as much again for the oracle's own order of operations.  The logits'
gradients are rounded to the logits' type once (eps / 2), after at most 2^-24 through fp32
and 64-bit sums, 2^-40 of scale * sum |dw|.
"""
import numpy as np
import pytest

import weight_only_int4_group_amd as w4
from oracle import block
from tests.gpu_helpers import note, to_dev, to_host, torch_cuda

pytestmark = pytest.mark.gpu

SCORE = {"softmax": w4.SCORE_SOFTMAX, "sigmoid": w4.SCORE_SIGMOID}
U = {"fp16": 2.0 ** -11, "bf16": 2.0 ** -8, "fp32": 2.0 ** -24}


def logits_of(T, E, dtype, seed, grid=0):
    torch = torch_cuda()
    x = np.random.default_rng([23, T, E, seed]).standard_normal((T, E)).astype(np.float32) * 2
    if grid:
        x = np.round(x * grid) / grid      # many ties
    t = torch.from_numpy(x).to({"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}[dtype])
    return t.cuda(), t.double().numpy()


def check_route(t, v, k, bias=None, **options):
    torch = torch_cuda()
    note(f"route {tuple(v.shape)} {t.dtype} k={k} bias={bias is not None} {options}")
    routing = w4.Routing(k, **{**options, "score": SCORE[options.get("score", "softmax")]})
    ids, weights = w4.w4a16_route(t, routing, None if bias is None else to_dev(bias))
    torch.cuda.synchronize()
    ref_ids, ref_w = block.route(v, k, bias=bias, **options)
    got = to_host(ids)
    assert np.array_equal(got, ref_ids), np.argwhere(got != ref_ids)[:5]
    w = to_host(weights).astype(np.float64)
    assert (np.abs(w - ref_w) <= 2.0 ** -23 * np.abs(ref_w) + 2.0 ** -149).all()
    dw = np.random.default_rng(k).standard_normal(ref_w.shape).astype(np.float32)
    d = w4.w4a16_route_backward(to_dev(dw), t, ids, routing)
    assert d.dtype == t.dtype
    ref = block.route_backward(dw.astype(np.float64), v, ref_ids, **options)
    u = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}[t.dtype]
    scale = abs(options.get("scale", 1.0)) * np.abs(dw).sum(1, keepdims=True)
    tiny = 2.0 ** -25 if t.dtype == torch.float16 else 0.0
    torch.cuda.synchronize()
    off = np.abs(d.double().cpu().numpy() - ref)
    assert (off <= (u + 2.0 ** -24) * np.abs(ref) + 2.0 ** -40 * scale + tiny).all()
    return ids, weights


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (3, 2, 2), (1, 8, 2), (5, 7, 3), (9, 64, 8), (6, 65, 4), (5, 128, 8),
                                   (5, 200, 6), (4, 256, 8), (3, 385, 10), (3, 1000, 16), (2, 1024, 64)])
def test_sizes(T, E, k, score, dtype):
    t, v = logits_of(T, E, dtype, 1)
    for renormalize in (True, False):
        check_route(t, v, k, score=score, renormalize=renormalize, scale=1.5)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups,topk_groups,k", [(8, 4, 2, 3), (64, 8, 3, 8), (256, 8, 4, 8), (60, 5, 2, 6),
                                                    (64, 64, 5, 5), (384, 3, 1, 8), (1024, 32, 4, 16), (6, 2, 2, 4)])
def test_groups_and_bias(E, groups, topk_groups, k, score):
    t, v = logits_of(7, E, "fp32", 2)
    bias = (np.random.default_rng(E).standard_normal(E) * 0.2).astype(np.float32)
    for b in (None, bias):
        check_route(t, v, k, b, score=score, groups=groups, topk_groups=topk_groups, scale=2.5)
    check_route(t, v, k, bias, score=score, renormalize=False)


@pytest.mark.parametrize("E,groups,topk_groups,k", [(192, 64, 3, 6), (320, 64, 63, 20), (576, 64, 1, 4), (130, 2, 1, 5)])
def test_lanes_past_the_last_group(E, groups, topk_groups, k):
    """A wave has more lanes than experts, whose group would be the 64th and more."""
    t, v = logits_of(5, E, "fp32", 9)
    bias = (np.random.default_rng(E).standard_normal(E) * 0.2).astype(np.float32)
    for b in (None, bias):
        for score in ("softmax", "sigmoid"):
            check_route(t, v, k, b, score=score, groups=groups, topk_groups=topk_groups)


@pytest.mark.parametrize("E", [16, 100, 512])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_ties_go_to_the_lowest_index(E, dtype):
    t, v = logits_of(40, E, dtype, 3, grid=1)
    check_route(t, v, 8)
    check_route(t, v, 8, score="sigmoid", groups=4, topk_groups=2)
    check_route(t, v, 8, np.zeros(E, np.float32))
    z = torch_cuda().zeros(3, E, device="cuda")
    ids, _ = check_route(z, np.zeros((3, E)), 8)
    assert to_host(ids).tolist() == [list(range(8))] * 3


@pytest.mark.parametrize("E", [8, 70, 300])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_masks_infinities_and_nan(E, score):
    torch = torch_cuda()
    t, v = logits_of(12, E, "fp32", 4)
    bias = np.linspace(-1, 1, E).astype(np.float32)
    t[0] = -float("inf")
    t[1, :] = -float("inf")
    t[1, E // 2] = -3.0
    t[2, ::2] = -float("inf")
    t[3, 1] = float("nan")
    t[4, 2] = float("inf")
    t[5, 2:4] = float("inf")
    t[6] = float("nan")
    t[7] = torch.finfo(torch.float32).min
    t[8] = t[8] * 1e4                     # scores that underflow
    t[9, :E - 2] = float("nan")
    v = t.double().cpu().numpy()
    for b in (None, bias):
        for renormalize in (True, False):
            check_route(t, v, 4, b, score=score, renormalize=renormalize)
    if E % 2 == 0:
        check_route(t, v, 4, score=score, groups=2, topk_groups=1)


def test_choices_that_32_bits_would_confuse():
    """Two experts whose biased scores differ by less than a step of fp32: logits x and 0 with the
    bias of the second one fp32 value above or below sigmoid(x) - 1 / 2."""
    rng = np.random.default_rng(9)
    x = rng.standard_normal(64).astype(np.float32)
    rows = np.full((64, 4), -9.0, np.float32)
    rows[:, 1], rows[:, 2] = x, 0.0
    torch = torch_cuda()
    s = 1 / (1 + np.exp(-x.astype(np.float64)))
    for i in range(64):
        b = np.float32(s[i] - 0.5)
        for bb in (b, np.nextafter(b, np.float32(9)), np.nextafter(b, np.float32(-9))):
            bias = np.array([0, 0, bb, 0], np.float32)
            ids, _ = w4.w4a16_route(to_dev(rows[i:i + 1]), w4.Routing(1, score=w4.SCORE_SIGMOID), to_dev(bias))
            gap = s[i] - (0.5 + np.float64(bb))
            assert abs(gap) < 2.0 ** -50 or int(ids[0, 0]) == (1 if gap > 0 else 2)
    torch.cuda.synchronize()


def test_many_tokens():
    t, v = logits_of(2049, 128, "bf16", 5)
    check_route(t, v, 8)
    torch = torch_cuda()
    big = torch.randn(1 << 17, 8, device="cuda", generator=torch.Generator("cuda").manual_seed(2))
    ids, w = w4.w4a16_route(big, w4.Routing(2))
    want = torch.sort(big, dim=1, descending=True, stable=True).indices[:, :2].int()
    assert torch.equal(ids, want)


def test_backward_skips_ids_out_of_range_and_adds_double_ones():
    torch = torch_cuda()
    t, v = logits_of(4, 70, "fp32", 6)
    ids = np.array([[0, -1, 69], [70, 3, 3], [-5, -1, 1000], [1 << 30, 2, 1]], np.int32)
    dw = np.random.default_rng(1).standard_normal((4, 3)).astype(np.float32)
    for score in ("softmax", "sigmoid"):
        for renormalize in (True, False):
            r = w4.Routing(3, score=SCORE[score], renormalize=renormalize)
            d = w4.w4a16_route_backward(to_dev(dw), t, to_dev(ids), r)
            ref = block.route_backward(dw.astype(np.float64), v, ids, score, renormalize)
            torch.cuda.synchronize()
            off = np.abs(d.double().cpu().numpy() - ref)
            assert (off <= 2.0 ** -23 * np.abs(ref) + 2.0 ** -40 * np.abs(dw).sum(1, keepdims=True)).all()


def test_backward_against_differences():
    torch = torch_cuda()
    t, v = logits_of(3, 24, "fp32", 7)
    for score in ("softmax", "sigmoid"):
        for renormalize in (True, False):
            r = w4.Routing(4, score=SCORE[score], renormalize=renormalize, scale=2.0)
            ids, w = w4.w4a16_route(t, r)
            dw = torch.randn(3, 4, device="cuda", generator=torch.Generator("cuda").manual_seed(3))
            d = w4.w4a16_route_backward(dw, t, ids, r)
            for e in (int(ids[1, 0]), int(ids[1, 3]), 23):
                # step 2^-10 (the choice holds: weights are in [0, 2], fp32): rounding 8 * 2^-24 * 4 |dw| / 2^-9,
                # third derivative below 2 * 2^-20
                a, b = t.clone(), t.clone()
                a[1, e] += 2.0 ** -10
                b[1, e] -= 2.0 ** -10
                (ia, wa), (ib, wb) = w4.w4a16_route(a, r), w4.w4a16_route(b, r)
                if not (torch.equal(ia, ids) and torch.equal(ib, ids)):
                    continue
                est = float(((wa - wb).double() * dw.double()).sum()) / float(a[1, e].double() - b[1, e].double())
                assert abs(est - float(d[1, e])) <= 8 * 2.0 ** -24 * 2 * float(dw.abs().sum()) * 2 ** 9 + 1e-5


def test_graph_and_streams():
    torch = torch_cuda()
    t, _ = logits_of(50, 160, "bf16", 8)
    bias = torch.randn(160, device="cuda") * 0.1
    r = w4.Routing(6, groups=8, topk_groups=3)
    ids, w = torch.empty(50, 6, dtype=torch.int32, device="cuda"), torch.empty(50, 6, device="cuda")
    dw, d = torch.randn(50, 6, device="cuda"), torch.empty_like(t)
    fwd, bwd = w4.RouteCall(t, r, ids, w, bias), w4.RouteBackwardCall(dw, t, ids, r, d)
    fwd()
    bwd()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        fwd()
        bwd()
    for i in range(4):
        t.copy_(t.roll(7, 1))
        fwd()
        bwd()
        want = [x.clone() for x in (ids, w, d)]
        ids.fill_(-3)
        w.zero_()
        d.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((ids, w, d), want)), f"replay {i}"
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        a = w4.w4a16_route(t, r, bias)
    side.synchronize()
    assert torch.equal(a[0], want[0]) and torch.equal(a[1], want[1])
