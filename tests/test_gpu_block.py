"""The expert feed-forward block's operators in a row, as a layer uses them: the residual addition and norms
after attention, the router, the experts, the next addition and norm; and back.

Tolerances.  The fp64 oracle runs the same chain twice, exactly and with every tensor that one operator hands
to the next rounded to the activations' type.  What the operators round inside them besides (the experts' H, dG
and dU, and the weights of the backward products) is at most as many roundings of the same size again, so a
result may be off by three times the distance between the two runs (relative L2; at least two roundings of its own).
"""
import numpy as np
import pytest

import weight_only_int4_group_amd as w4
from oracle import block
from tests.gpu_helpers import note, to_dev, torch_cuda
from tests.test_gpu_experts import stack, tensor, unit

pytestmark = pytest.mark.gpu

EPS = 1e-6
ROUTINGS = {
    "softmax": dict(k=2),
    "sigmoid": dict(k=3, score="sigmoid", bias=True, groups=4, topk_groups=2, scale=2.5),
}


class Layer:
    """Inputs, parameters and upstream gradients of one block, on the device and in fp64."""

    def __init__(self, T, dtype, kind, D=256, N=384, E=8):
        self.T, self.D, self.E, self.dtype = T, D, E, dtype
        names = ("x", "y", "dr2", "dh2")
        self.dev, self.host = {}, {}
        for i, n in enumerate(names):
            self.dev[n], self.host[n] = tensor(dtype, 31 + i, T, D)
        rng = np.random.default_rng([83, T, D, E])
        norms = {n: 1 + 0.2 * rng.standard_normal(D) for n in ("post", "pre", "next")}
        for n, v in norms.items():
            t = to_dev(v.astype(np.float32)).to(self.dev["x"].dtype)
            self.dev[n], self.host[n] = w4.Norm(w4.NORM_RMS, weight=t, eps=EPS), ("rms", t.double().cpu().numpy(), None, EPS)
        t = to_dev(rng.standard_normal((-(-T // 16), D)).astype(np.float32)).to(self.dev["x"].dtype)
        self.dev["gate"], self.host["gate"] = t, t.double().cpu().numpy()
        self.Wr = rng.standard_normal((D, E)) / np.sqrt(D)
        self.bias = 0.1 * rng.standard_normal(E).astype(np.float32)
        self.stacks = stack(1, E, N, D), stack(2, E, N, D), stack(3, E, D, N)
        opt = dict(ROUTINGS[kind])
        self.with_bias = opt.pop("bias", False)
        self.opt = opt
        self.routing = w4.Routing(**{**opt, "score": getattr(w4, "SCORE_" + opt.get("score", "softmax").upper())})
        self.pad = np.arange(T) % 13 == 12     # padded tokens: no expert

    def gpu(self):
        """(forward results, backward results)"""
        torch, d = torch_cuda(), self.dev
        Wr = to_dev(self.Wr.astype(np.float32))
        gate = dict(gate=d["gate"], gate_rows=16)
        r1, h1 = w4.w4a16_norm_block(d["x"], d["y"], d["post"], d["pre"], **gate)
        logits = h1.float() @ Wr
        logits[to_dev(self.pad)] = -float("inf")
        ids, w = w4.w4a16_route(logits, self.routing, to_dev(self.bias) if self.with_bias else None)
        N = self.stacks[0].dev.N
        pre = tuple(torch.empty(self.T, self.routing.k, N, dtype=h1.dtype, device="cuda") for _ in range(2))
        Y = w4.w4a16_experts(h1, ids, w, *(s.dev for s in self.stacks), preact=pre)
        r2, h2 = w4.w4a16_norm_block(r1, Y, None, d["next"])
        dr1, dY, g2 = w4.w4a16_norm_block_backward(d["dr2"], d["dh2"], Y, r2, None, d["next"])
        dh1, dw = w4.w4a16_experts_backward(dY, ids, w, *pre, *(s.transposed() for s in self.stacks))
        dl = w4.w4a16_route_backward(dw, logits, ids, self.routing)
        dh1 = (dh1.float() + dl @ Wr.T).to(h1.dtype)
        dx, dy, g1 = w4.w4a16_norm_block_backward(dr1, dh1, d["y"], r1, d["post"], d["pre"], **gate)
        return ids, dict(r2=r2, h2=h2, dx=dx, dy=dy, dgate=g1.gate, dpost=g1.post_weight, dpre=g1.pre_weight,
                         dnext=g2.pre_weight, dlogits=dl)

    def forward(self, x, ids=None, q=lambda v: v):
        h, W = self.host, [s.W for s in self.stacks]
        r1, h1 = (q(v) for v in block.norm_block(x, h["y"], h["post"], h["pre"], h["gate"], 16))
        logits = np.where(self.pad[:, None], -np.inf, h1 @ self.Wr)
        own, w = block.route(logits, bias=self.bias if self.with_bias else None, **self.opt)
        if ids is not None:                    # the choice that was made, its weights from these logits
            s = block.scores(logits, self.opt.get("score", "softmax"))
            w = np.where(ids >= 0, np.take_along_axis(s, np.maximum(ids, 0), 1), 0.0)
            w = self.opt.get("scale", 1.0) * np.divide(w, w.sum(1, keepdims=True), out=np.zeros_like(w),
                                                       where=ids >= 0)
            own = ids
        Y, G, U = block.experts(h1, own, w, *W)
        Y, G, U = q(Y), q(G), q(U)
        r2, h2 = (q(v) for v in block.norm_block(r1, Y, pre=h["next"]))
        return dict(r1=r1, h1=h1, logits=logits, ids=own, w=w, Y=Y, G=G, U=U, r2=r2, h2=h2)

    def both(self, ids, q=lambda v: v):
        h, W, f = self.host, [s.W for s in self.stacks], self.forward(self.host["x"], ids, q)
        b2 = block.norm_block_backward(h["dr2"], h["dh2"], f["Y"], f["r2"], pre=h["next"])
        dr1, dY = q(b2["dx"]), q(b2["dy"])
        dh1, dw = block.experts_backward(dY, f["ids"], f["w"], f["G"], f["U"], *W)
        dl = block.route_backward(dw, f["logits"], f["ids"], **{k: v for k, v in self.opt.items() if k != "k"})
        dh1 = q(q(dh1) + dl @ self.Wr.T)
        b1 = block.norm_block_backward(dr1, dh1, h["y"], f["r1"], h["post"], h["pre"], h["gate"], 16)
        return dict(r2=f["r2"], h2=f["h2"], dx=q(b1["dx"]), dy=q(b1["dy"]), dgate=b1["gate"], dpost=b1["post_weight"],
                    dpre=b1["pre_weight"], dnext=b2["pre_weight"], dlogits=dl)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("kind", sorted(ROUTINGS))
@pytest.mark.parametrize("T", [1, 37, 200])
def test_layer_forward_and_backward(T, kind, dtype):
    torch = torch_cuda()
    note(f"block T={T} {kind} {dtype}")
    layer = Layer(T, dtype, kind)
    ids, got = layer.gpu()
    ids = ids.cpu().numpy()
    assert (ids[layer.pad] == -1).all() and (ids[~layer.pad] >= 0).all()
    dt = layer.dev["x"].dtype
    exact = layer.both(ids)
    rounded = layer.both(ids, lambda v: torch.from_numpy(v).to(dt).double().numpy())
    for n, t in got.items():
        v, ref = t.double().cpu().numpy(), exact[n]
        size = np.linalg.norm(ref)
        bound = 3 * np.linalg.norm(rounded[n] - ref) + 2 * unit(dtype) * size
        err = np.linalg.norm(v - ref)
        assert err <= bound, f"{n}: {err / size:.3g} of its norm, bound {bound / size:.3g}"
    # the gradient of x against differences of the forward pass, the experts as chosen
    def loss(x):
        f = layer.forward(x, ids)
        return (f["r2"] * layer.host["dr2"]).sum() + (f["h2"] * layer.host["dh2"]).sum()
    v = np.random.default_rng([89, T]).standard_normal((T, layer.D))
    step = 1e-5
    diff = (loss(layer.host["x"] + step * v) - loss(layer.host["x"] - step * v)) / (2 * step)
    far = 3 * np.linalg.norm(rounded["dx"] - exact["dx"]) + 2 * unit(dtype) * np.linalg.norm(exact["dx"])
    assert abs((exact["dx"] * v).sum() - diff) <= 1e-6 * (abs(diff) + np.linalg.norm(exact["dx"]) * np.linalg.norm(v))
    assert abs((got["dx"].double().cpu().numpy() * v).sum() - diff) <= 1.01 * far * np.linalg.norm(v)


def test_layer_in_a_graph_and_two_at_once():
    """The prepared calls of two layers, captured together on two streams and replayed with other inputs, give the
    bits of the same calls run one by one."""
    torch = torch_cuda()
    note("block in a graph")
    chains = []
    for T in (5, 90):
        layer = Layer(T, "bf16", "softmax")
        d, k, N, E, D = layer.dev, layer.routing.k, layer.stacks[0].dev.N, layer.E, layer.D

        def empty(*s, dtype=d["x"].dtype):
            return torch.zeros(*s, dtype=dtype, device="cuda")
        r1, h1, Y, r2, h2, dr1, dY, dh1, dx, dy = (empty(T, D) for _ in range(10))
        logits, dl = (empty(T, E, dtype=torch.float32) for _ in range(2))
        logits.normal_()
        ids, w, dw = empty(T, k, dtype=torch.int32), *(empty(T, k, dtype=torch.float32) for _ in range(2))
        G, U = empty(T, k, N), empty(T, k, N)
        g1, g2 = w4.NormGrads(pre_weight=empty(D, dtype=torch.float32)), w4.NormGrads(pre_weight=empty(D, dtype=torch.float32))
        dev = [s.dev for s in layer.stacks]
        calls = [w4.NormBlockCall(d["x"], d["y"], r1, h1, d["post"], d["pre"]),
                 w4.RouteCall(logits, layer.routing, ids, w),
                 w4.ExpertsCall(h1, ids, w, *dev, Y, preact=(G, U)),
                 w4.NormBlockCall(r1, Y, r2, h2, None, d["next"]),
                 w4.NormBlockBackwardCall(d["dr2"], d["dh2"], Y, r2, dr1, dY, g2, None, d["next"]),
                 w4.ExpertsBackwardCall(dY, ids, w, G, U, *(s.transposed() for s in layer.stacks), dh1, dw),
                 w4.RouteBackwardCall(dw, logits, ids, layer.routing, dl),
                 w4.NormBlockBackwardCall(dr1, dh1, d["y"], r1, dx, dy, g1, d["post"], d["pre"])]
        chains.append((calls, (d["x"], logits), (r2, h2, dx, dy, dl, g1.pre_weight, g2.pre_weight)))
    torch.cuda.synchronize()

    def eager():
        for calls, _, outs in chains:
            for c in calls:
                c()
        torch.cuda.synchronize()
        return [o.clone() for _, _, outs in chains for o in outs]
    eager()
    main, side = torch.cuda.Stream(), torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=main):
        side.wait_stream(main)
        for c in chains[0][0]:
            c()
        with torch.cuda.stream(side):
            for c in chains[1][0]:
                c()
        main.wait_stream(side)
    for i in range(4):
        for _, inputs, _ in chains:
            for t in inputs:
                t.mul_(-0.9)                  # another routing on every replay
        want = eager()
        for _, _, outs in chains:
            for o in outs:
                o.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((o for _, _, outs in chains for o in outs), want)), f"replay {i}"
