"""Measured cases of the expert feed-forward block's operators, with their plain forms.

T tokens of width D, E experts of inner width N, top-k of them chosen per token.  Activations
are fp16 or bf16.

  norm             r = alpha * x + gate * post(y),  h = pre(r)
                   post and pre: RMS norm, layer norm or none; y the block's output, x the
                   residual stream; gate one vector, or one per `gate_rows` tokens
  norm_backward    R = dr + (gradient of pre at r)(dh),  dx = alpha * R,
                   dy = (gradient of post at y)(gate * R),  and the fp32 gradients of the gate
                   and of the norms' weights and biases
  route            scores of logits [T][E] (softmax or sigmoid); the choice goes by score + bias,
                   within the best `topk_groups` of `groups` groups (a group's value is the sum
                   of its two best); ties to the lowest index.  Weights are the chosen scores,
                   renormalised or not, times `scale`
  route_backward   gradient of the logits from that of the weights
  experts          Y = residual + sum over the chosen experts e of w_e * (act(G) * U) . Wd_e^T,
                   G = X . Wg_e^T,  U = X . Wu_e^T   (G and U returned when training)
  experts_backward from dY and the kept G and U: dX and the gradients of the routing weights

The experts' weights are in this library's packed layout (include/w4a16.h), one expert after
the other: W_hat[n][k] = (q - z) * scale, times an optional per-input-channel fp16 scale: s[D]
for gate and up, s_down[E][N] for down.  They are frozen, so only activations have gradients.
"""
import math

import torch

own = False

GROUP = 128
DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
ACTS = ("silu", "gelu", "gelu_tanh", "relu")
KINDS = ("none", "rms", "layer")
EPS = 1e-5


def _norm(name, op, T, D, dtype, post="none", pre="rms", y=True, gate=0, alpha=1.0):
    """gate: 0 none, else the tokens that share one gate vector."""
    return {"name": name, "op": op, "T": T, "D": D, "dtype": dtype, "post": post, "pre": pre, "y": y,
            "gate": gate, "alpha": alpha}


def _route(name, op, T, E, k, dtype, score="softmax", bias=False, groups=1, topk_groups=1,
           renormalize=True, scale=1.0):
    return {"name": name, "op": op, "T": T, "E": E, "k": k, "dtype": dtype, "score": score,
            "bias": bias, "groups": groups, "topk_groups": topk_groups, "renormalize": renormalize,
            "scale": scale}


def _experts(name, op, T, E, k, D, N, dtype, act="silu", s=False, residual=False, train=False,
             skip=0.0):
    """skip: the share of slots that name no expert (padded tokens, experts held elsewhere)."""
    return {"name": name, "op": op, "T": T, "E": E, "k": k, "D": D, "N": N, "dtype": dtype,
            "act": act, "s": s, "residual": residual, "train": train, "skip": skip}


def listed():
    return [
        # decode of one token, 8B width: the residual addition and the next block's norm
        _norm("norm_decode", "norm", 1, 4096, "fp16"),
        # batched decode, 7B width: norms on both sides, a gate vector, a residual scale
        _norm("norm_batched", "norm", 64, 3584, "bf16", post="rms", gate=64, alpha=0.5),
        # prefill of 4096 tokens, 70B width: norms on both sides of the block
        _norm("norm_prefill", "norm", 4096, 8192, "bf16", post="rms"),
        # training, 8B width, four sequences of odd length with a gate each, layer norms
        _norm("norm_bwd", "norm_backward", 4 * 1023, 4096, "bf16", post="layer", pre="layer",
              gate=1023, alpha=0.75),
        # decode of one token, 64 experts
        _route("route_decode", "route", 1, 64, 8, "fp32"),
        # prefill, 256 experts in groups, chosen with a balancing bias
        _route("route_prefill", "route", 8192, 256, 8, "fp32", score="sigmoid", bias=True, groups=8,
               topk_groups=4, scale=2.5),
        # training: back through the router of 128 experts
        _route("route_bwd", "route_backward", 4096, 128, 8, "bf16"),
        # decode of one token, 8 experts of the 8B layer's feed-forward size
        _experts("experts_decode", "experts", 1, 8, 2, 4096, 14336, "bf16", residual=True),
        # batched decode over many small experts
        _experts("experts_batched", "experts", 64, 64, 8, 4096, 1024, "fp16"),
        # prefill of 4096 tokens over many small experts
        _experts("experts_prefill", "experts", 4096, 64, 8, 4096, 1024, "bf16", residual=True),
        # training forward, odd length, input-channel scales, G and U kept
        _experts("experts_train", "experts", 1531, 16, 4, 3584, 2560, "fp16", act="gelu", s=True,
                 train=True),
        # adapter training: back through 8 experts of the 8B layer's feed-forward size
        _experts("experts_bwd", "experts_backward", 2048, 8, 2, 4096, 14336, "bf16",
                 residual=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("norm", "norm_backward", "route", "route_backward", "experts",
                     "experts_backward"))
    dtype = rng.choice(("fp16", "bf16"))
    while True:
        T = _log(rng, 1, 8192)
        if op.startswith("norm"):
            unit = rng.choice((1, 8, 128))
            D = unit * _log(rng, max(1, 16 // unit), 16384 // unit)
            if T * D > 4096 * 8192:
                continue
            backward = op == "norm_backward"
            post = rng.choice(KINDS)
            pre = rng.choice(KINDS[1:] if post == "none" else KINDS)
            case = _norm(None, op, T, D, dtype, post, pre, y=backward or post != "none" or rng.random() < 0.7,
                         gate=rng.choice((0, T, _log(rng, 1, T))), alpha=rng.choice((1.0, 0.5, 1.7)))
            case["gate"] *= case["y"]
        elif op.startswith("route"):
            groups = rng.choice((1, 1, 2, 4, 8))
            E = groups * max(2, _log(rng, 2, 512) // groups)
            topk_groups = rng.randint(1, groups)
            k = rng.randint(1, min(16, E // groups * topk_groups))
            case = _route(None, op, T, E, k, rng.choice(("fp32", "fp16", "bf16")),
                          rng.choice(("softmax", "sigmoid")), rng.random() < 0.5, groups, topk_groups,
                          rng.random() < 0.7, rng.choice((1.0, 2.5)))
        else:
            E = _log(rng, 1, 128)
            k = rng.randint(1, min(8, E))
            D, N = 128 * _log(rng, 1, 64), 128 * _log(rng, 1, 112)
            if T * k * D * N > 2048 * 2 * 4096 * 14336 or E * D * N > 8 * 4096 * 14336:
                continue
            train = op == "experts" and rng.random() < 0.3
            case = _experts(None, op, T, E, k, D, N, dtype, rng.choice(ACTS), rng.random() < 0.4,
                            rng.random() < 0.5, train, 0.0 if train else rng.choice((0.0, 0.0, 0.3)))
        del case["name"]
        return case


# ---- inputs -----------------------------------------------------------------------------

def _packed(gen, E, N, K):
    """E packed weights [N][K] of about N(0, 1/K): code bytes, scales and zero points."""
    codes = torch.empty(E * N * K // 2, dtype=torch.uint8, device="cuda")
    for part in codes.view(E, -1):
        q = torch.empty(2, part.numel(), dtype=torch.float16, device="cuda")
        q = q.normal_(7.5, 2.6, generator=gen).round_().clamp_(0, 15).to(torch.uint8)
        part.copy_(q[0] | (q[1] << 4))
    G = K // GROUP
    Gq = (G + 3) // 4
    shape = (E, Gq, N // 16, 16, 4)
    scales = (torch.rand(shape, generator=gen, device="cuda") * 0.4 + 0.8) / (2.6 * math.sqrt(K))
    zeros = torch.randint(7, 9, shape, generator=gen, device="cuda")
    # the last quad's slots past K / 128 groups are zero
    keep = (torch.arange(4 * Gq, device="cuda") < G).view(1, Gq, 1, 1, 4)
    return codes, (scales * keep).half().view(-1), (zeros * keep).half().view(-1)


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    dt, op, T = DTYPES[case["dtype"]], case["op"], case["T"]

    def normal(*shape, std=1.0, mean=0.0, dtype=dt):
        return (torch.randn(*shape, generator=gen, device="cuda") * std + mean).to(dtype)

    st = {"case": case}
    if op.startswith("norm"):
        D = case["D"]
        for which in ("post", "pre"):
            kind = case[which]
            st[which] = (None if kind == "none" else normal(D, std=0.2, mean=1.0),
                         normal(D, std=0.2) if kind == "layer" else None)
        y = normal(T, D, std=3.0, mean=0.5) if case["y"] else None
        gate = normal(-(-T // case["gate"]), D, std=0.5) if case["gate"] else None
        st |= {"y": y, "gate": gate}
        if op == "norm":
            st["x"] = normal(T, D, std=2.0)
        else:
            st |= {"r": normal(T, D, std=2.0), "dr": normal(T, D, std=0.1),
                   "dh": normal(T, D, std=0.1) if case["pre"] != "none" else None}
    elif op.startswith("route"):
        E = case["E"]
        st["logits"] = normal(T, E, std=1.5)
        st["bias"] = normal(E, std=0.1, dtype=torch.float32) if case["bias"] else None
        if op == "route_backward":
            st["ids"] = _choose(st["logits"], st["bias"], case)[0]
            st["dweights"] = normal(T, case["k"], dtype=torch.float32)
    else:
        E, k, D, N = case["E"], case["k"], case["D"], case["N"]
        # distinct experts per token, some in more demand than others
        demand = torch.rand(E, generator=gen, device="cuda").log()[None] * 0.3
        noise = -torch.rand(T, E, generator=gen, device="cuda").clamp(min=1e-9).log()
        order = torch.argsort(noise.log() - demand, dim=1, stable=True)
        ids = order[:, :k].to(torch.int32)
        skip = torch.rand(T, k, generator=gen, device="cuda") < case["skip"]
        st["ids"] = torch.where(skip, -1, ids).contiguous()
        w = torch.rand(T, k, generator=gen, device="cuda") + 0.2
        st["weights"] = w / w.sum(1, keepdim=True)
        for name, n, c in (("gate", N, D), ("up", N, D), ("down", D, N)):
            st[name] = _packed(gen, E, n, c)
        st["s"] = st["s_down"] = None
        if case["s"]:
            st["s"] = torch.exp(0.5 * torch.randn(D, generator=gen, device="cuda")).half()
            st["s_down"] = torch.exp(0.5 * torch.randn(E, N, generator=gen, device="cuda")).half()
        if op == "experts":
            st["X"] = normal(T, D)
            st["residual"] = normal(T, D) if case["residual"] else None
        else:
            st |= {"G": normal(T, k, N), "U": normal(T, k, N), "dY": normal(T, D, std=0.1),
                   "add": normal(T, D, std=0.1) if case["residual"] else None}
    if own:
        st["call"] = _own_call(st)
    return st


def _own_call(st):
    """The prepared call a user's program keeps: packed weights, output buffers, workspace."""
    import weight_only_int4_group_amd as w4
    case = st["case"]
    dt, op, T = DTYPES[case["dtype"]], case["op"], case["T"]

    def empty(*shape, dtype=dt):
        return torch.empty(*shape, dtype=dtype, device="cuda")

    if op.startswith("norm"):
        D = case["D"]
        norms = {}
        for which in ("post", "pre"):
            w, b = st[which]
            kind = getattr(w4, "NORM_" + case[which].upper())
            norms[which] = w4.Norm(kind, weight=w, bias=b, eps=EPS) if w is not None else None
        options = {"gate": st["gate"], "gate_rows": case["gate"], "alpha": case["alpha"]}
        if op == "norm":
            r = empty(T, D) if st["y"] is not None else None
            h = empty(T, D) if norms["pre"] else None
            outs = [t for t in (r, h) if t is not None]
            return w4.NormBlockCall(st["x"], st["y"], r, h, **norms, **options), outs
        f32 = torch.float32
        grads = w4.NormGrads(
            gate=empty(*st["gate"].shape, dtype=f32) if st["gate"] is not None else None,
            post_weight=empty(D, dtype=f32) if norms["post"] else None,
            post_bias=empty(D, dtype=f32) if case["post"] == "layer" else None,
            pre_weight=empty(D, dtype=f32) if norms["pre"] else None,
            pre_bias=empty(D, dtype=f32) if case["pre"] == "layer" else None)
        dx, dy = empty(T, D), empty(T, D)
        call = w4.NormBlockBackwardCall(st["dr"], st["dh"], st["y"], st["r"], dx, dy, grads=grads,
                                        **norms, **options)
        outs = [dx, dy, grads.gate, grads.post_weight, grads.post_bias, grads.pre_weight,
                grads.pre_bias]
        return call, [t for t in outs if t is not None]
    if op.startswith("route"):
        k = case["k"]
        routing = w4.Routing(k, score=getattr(w4, "SCORE_" + case["score"].upper()),
                             groups=case["groups"], topk_groups=case["topk_groups"],
                             renormalize=case["renormalize"], scale=case["scale"])
        if op == "route":
            ids, weights = empty(T, k, dtype=torch.int32), empty(T, k, dtype=torch.float32)
            return w4.RouteCall(st["logits"], routing, ids, weights, bias=st["bias"]), [ids, weights]
        dlogits = empty(T, case["E"])
        call = w4.RouteBackwardCall(st["dweights"], st["logits"], st["ids"], routing, dlogits)
        return call, [dlogits]
    E, k, D, N = case["E"], case["k"], case["D"], case["N"]
    act = getattr(w4, "ACT_" + case["act"].upper())
    packed = {name: w4.PackedExperts(*st[name], E, n, c)
              for name, n, c in (("gate", N, D), ("up", N, D), ("down", D, N))}
    if op == "experts":
        Y = empty(T, D)
        saved = [empty(T, k, N), empty(T, k, N)] if case["train"] else []
        call = w4.ExpertsCall(st["X"], st["ids"], st["weights"], packed["gate"], packed["up"],
                              packed["down"], Y, s=st["s"], s_down=st["s_down"], act=act,
                              residual=st["residual"], preact=tuple(saved) or None)
        return call, [Y] + saved
    transposed = [w4.w4a16_transpose_experts(packed[name]) for name in ("gate", "up", "down")]
    dX, dw = empty(T, D), empty(T, k)
    call = w4.ExpertsBackwardCall(st["dY"], st["ids"], st["weights"], st["G"], st["U"], *transposed,
                                  dX, dw, s=st["s"], s_down=st["s_down"], act=act, add=st["add"])
    return call, [dX, dw]


# ---- plain forms -------------------------------------------------------------------------

def _normalize(v, kind):
    """(normalised v, 1 / its deviation)"""
    if kind == "layer":
        v = v - v.mean(1, keepdim=True)
    inv = 1 / torch.sqrt((v * v).mean(1, keepdim=True) + EPS)
    return v * inv, inv


def _affine(n, weight, bias):
    n = n * weight.float()
    return n if bias is None else n + bias.float()


def _normalize_backward(d, n, inv, kind):
    d = d - n * (d * n).mean(1, keepdim=True) if kind == "rms" else \
        d - d.mean(1, keepdim=True) - n * (d * n).mean(1, keepdim=True)
    return d * inv


def _plain_norm(st):
    case = st["case"]
    dt, T = DTYPES[case["dtype"]], case["T"]
    gate = None
    if st["gate"] is not None:
        gate = st["gate"].float().repeat_interleave(case["gate"], 0)[:T]
    if case["op"] == "norm":
        r = st["x"].float() * case["alpha"]
        outs = []
        if st["y"] is not None:
            y = st["y"].float()
            if case["post"] != "none":
                y = _affine(_normalize(y, case["post"])[0], *st["post"])
            r = r + (y if gate is None else gate * y)
            outs.append(r.to(dt))
        if case["pre"] != "none":
            outs.append(_affine(_normalize(r, case["pre"])[0], *st["pre"]).to(dt))
        return outs
    R = st["dr"].float()
    pre_grads, post_grads, dgate = [], [], []

    # sums over many rows, in 64 bits
    def column_sums(v):
        return v.sum(0, dtype=torch.float64).float()

    if case["pre"] != "none":
        dh = st["dh"].float()
        n, inv = _normalize(st["r"].float(), case["pre"])
        R = R + _normalize_backward(dh * st["pre"][0].float(), n, inv, case["pre"])
        pre_grads = [column_sums(dh * n)]
        if case["pre"] == "layer":
            pre_grads.append(column_sums(dh))
    y = st["y"].float()
    n, inv = (y, None) if case["post"] == "none" else _normalize(y, case["post"])
    if gate is not None:
        p = R * (n if case["post"] == "none" else _affine(n, *st["post"]))
        rows, B = case["gate"], st["gate"].shape[0]
        p = torch.nn.functional.pad(p, (0, 0, 0, B * rows - T))
        dgate = [p.view(B, rows, -1).sum(1, dtype=torch.float64).float()]
    dp = R if gate is None else R * gate
    if case["post"] == "none":
        dy = dp
    else:
        dy = _normalize_backward(dp * st["post"][0].float(), n, inv, case["post"])
        post_grads = [column_sums(dp * n)]
        if case["post"] == "layer":
            post_grads.append(column_sums(dp))
    return [(R * case["alpha"]).to(dt), dy.to(dt)] + dgate + post_grads + pre_grads


def _choose(logits, bias, case):
    """Chosen experts, in the order of their biased scores, and all scores, in 64 bits: a
    choice between two close scores is decided by what 32 bits round away."""
    l = logits.double()
    if case["score"] == "softmax":
        e = torch.exp(l - l.amax(1, keepdim=True))
        score = e / e.sum(1, keepdim=True)
    else:
        score = 1 / (1 + torch.exp(-l))
    rank = score if bias is None else score + bias.double()
    groups, T = case["groups"], l.shape[0]
    if groups > 1:
        best = rank.view(T, groups, -1).sort(dim=2, descending=True).values[:, :, :2].sum(2)
        order = best.sort(dim=1, descending=True, stable=True).indices[:, :case["topk_groups"]]
        kept = torch.zeros_like(best, dtype=torch.bool).scatter(1, order, True)
        kept = kept[:, :, None].expand(T, groups, rank.shape[1] // groups).reshape(rank.shape)
        rank = torch.where(kept, rank, -math.inf)
    ids = rank.sort(dim=1, descending=True, stable=True).indices[:, :case["k"]]
    return ids.to(torch.int32), score


def _plain_route(st):
    case, logits = st["case"], st["logits"]
    if case["op"] == "route":
        ids, score = _choose(logits, st["bias"], case)
        w = score.gather(1, ids.long())
        if case["renormalize"]:
            w = w / w.sum(1, keepdim=True)
        return [ids, (w * case["scale"]).float()]
    l, ids, dw = logits.float(), st["ids"].long(), st["dweights"] * case["scale"]
    if case["score"] == "softmax":
        e = torch.exp(l - l.amax(1, keepdim=True))
        score = e / e.sum(1, keepdim=True)
    else:
        score = 1 / (1 + torch.exp(-l))
    chosen = score.gather(1, ids)
    if case["renormalize"]:
        total = chosen.sum(1, keepdim=True)
        dw = (dw - (dw * chosen).sum(1, keepdim=True) / total) / total
    d = torch.zeros_like(l).scatter(1, ids, dw)
    if case["score"] == "softmax":
        d = score * (d - (d * score).sum(1, keepdim=True))
    else:
        d = d * score * (1 - score)
    return [d.to(logits.dtype)]


def _dequantized(w, e, E, N, K):
    """(q - z) * scale of expert e's weight [N][K] in fp32 from the packed buffers."""
    wq, scales, zeros = (v.view(E, -1)[e] for v in w)
    G, NB = K // GROUP, N // 16
    words = wq.view(torch.int32).view(G, NB, 4, 16, 4, 1)
    shift = torch.tensor([4 * (j // 2 + 4 * (j % 2)) for j in range(8)], dtype=torch.int32,
                         device=wq.device)
    q = ((words >> shift) & 15).permute(1, 3, 0, 4, 2, 5).reshape(N, G, GROUP).float()

    def rows(v):
        return v.view(-1, NB, 16, 4).permute(1, 2, 0, 3).reshape(N, -1)[:, :G].float()
    return ((q - rows(zeros)[..., None]) * rows(scales)[..., None]).view(N, K)


def _act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * torch.erfc(z * -math.sqrt(0.5))
    return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))


def _act_grad(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "silu":
        sig = 1 / (1 + torch.exp(-z))
        return sig * (1 + z * (1 - sig))
    if act == "gelu":
        return (0.5 * torch.erfc(z * -math.sqrt(0.5))
                + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi)))
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (z + 0.044715 * z * z * z))
    return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)


def _plain_experts(st):
    case = st["case"]
    dt, act, T, k = DTYPES[case["dtype"]], case["act"], case["T"], case["k"]
    E, D, N = case["E"], case["D"], case["N"]
    ids = st["ids"].view(-1)
    order = torch.argsort(ids, stable=True)
    counts = torch.bincount(ids + 1, minlength=E + 1).tolist()
    s = None if st["s"] is None else st["s"].float()
    scale = st["weights"].view(-1, 1)
    forward = case["op"] == "experts"
    source = (st["X"] if forward else st["dY"]).float()
    if forward and s is not None:
        source = source * s
    total = torch.zeros(T * k, D, device="cuda")
    if case["train"]:
        pre = torch.empty(2, T * k, N, dtype=dt, device="cuda")
    dw = torch.zeros(T * k, device="cuda")
    at = counts[0]
    for e in range(E):
        slots = order[at:at + counts[e + 1]]
        at += counts[e + 1]
        if not len(slots):
            continue
        gate, up, down = (_dequantized(st[name], e, E, n, c)
                          for name, n, c in (("gate", N, D), ("up", N, D), ("down", D, N)))
        if st["s_down"] is not None:
            down = down * st["s_down"][e].float()
        rows = source[slots // k]
        if forward:
            g, u = rows @ gate.t(), rows @ up.t()
            if case["train"]:
                pre[0, slots], pre[1, slots] = g.to(dt), u.to(dt)
            total[slots] = (_act(g, act) * u @ down.t()) * scale[slots]
        else:
            g, u = (st[n].view(T * k, N)[slots].float() for n in ("G", "U"))
            dh, a = rows @ down, _act(g, act)
            dw[slots] = (dh * a * u).sum(1)
            dh = dh * scale[slots]
            total[slots] = (dh * u * _act_grad(g, act)) @ gate + (dh * a) @ up
    y = total.view(T, k, D).sum(1)
    if not forward and s is not None:
        y = y * s
    extra = st["residual"] if forward else st["add"]
    if extra is not None:
        y = y + extra.float()
    if forward:
        return [y.to(dt)] + ([p.view(T, k, N) for p in pre] if case["train"] else [])
    return [y.to(dt), dw.view(T, k).to(dt)]


def run(state):
    if own:
        call, outs = state["call"]
        call()
        return outs
    op = state["case"]["op"]
    plain = (_plain_norm if op.startswith("norm") else
             _plain_route if op.startswith("route") else _plain_experts)
    return plain(state)


# ---- the definitions in 64 bits ------------------------------------------------------------

def _exact_norm(st):
    case, f64 = st["case"], torch.float64
    T = case["T"]

    def norm(v, kind, weight, bias):
        if kind == "none":
            return v
        if kind == "layer":
            var, mean = torch.var_mean(v, 1, correction=0, keepdim=True)
            v = (v - mean) * torch.rsqrt(var + EPS)
        else:
            v = v * torch.rsqrt(torch.mean(torch.square(v), 1, keepdim=True) + EPS)
        return weight * v + (0.0 if bias is None else bias)

    t = {n: None if st.get(n) is None else st[n].to(f64) for n in ("x", "y", "r", "dr", "dh", "gate")}
    params = {w: [None if v is None else v.to(f64) for v in st[w]] for w in ("post", "pre")}

    def per_token(g):
        return g[torch.arange(T, device="cuda") // case["gate"]]

    if case["op"] == "norm":
        r = case["alpha"] * t["x"]
        if t["y"] is not None:
            p = norm(t["y"], case["post"], *params["post"])
            r = r + (p if t["gate"] is None else per_token(t["gate"]) * p)
        outs = [r] if t["y"] is not None else []
        return outs + ([norm(r, case["pre"], *params["pre"])] if case["pre"] != "none" else [])
    # the gradients by automatic differentiation of the definition
    with torch.enable_grad():
        leaves = {n: t[n].requires_grad_() for n in ("y", "r", "gate") if t[n] is not None}
        named = {}
        for w in ("post", "pre"):
            for n, v in zip(("weight", "bias"), params[w]):
                if v is not None:
                    named[w, n] = v.requires_grad_()
        R = t["dr"]
        grads = {}
        if case["pre"] != "none":
            h = norm(leaves["r"], case["pre"], *params["pre"])
            wanted = [k for k in named if k[0] == "pre"]
            got = torch.autograd.grad(h, [leaves["r"]] + [named[k] for k in wanted], t["dh"])
            R = R + got[0]
            grads |= dict(zip(wanted, got[1:]))
        p = norm(leaves["y"], case["post"], *params["post"])
        if t["gate"] is not None:
            p = p * per_token(leaves["gate"])
        wanted = [k for k in named if k[0] == "post"]
        first = [leaves["y"]] + ([leaves["gate"]] if t["gate"] is not None else [])
        got = torch.autograd.grad(p, first + [named[k] for k in wanted], R)
        grads |= dict(zip(wanted, got[len(first):]))
    outs = [case["alpha"] * R, *got[:len(first)]]
    return outs + [grads[k] for k in (("post", "weight"), ("post", "bias"), ("pre", "weight"),
                                      ("pre", "bias")) if k in grads]


def _exact_route(st):
    case = st["case"]
    T, E, k = case["T"], case["E"], case["k"]
    l = st["logits"].double()
    if case["op"] == "route":
        score = torch.softmax(l, 1) if case["score"] == "softmax" else torch.special.expit(l)
        value = score if st["bias"] is None else score + st["bias"].double()
        if case["groups"] > 1:
            size = E // case["groups"]
            best = torch.topk(value.view(T, -1, size), min(2, size), 2).values.sum(2)
            border = torch.topk(best, case["topk_groups"], 1).values[:, -1:]
            value = torch.where((best >= border).repeat_interleave(size, 1), value, -math.inf)
        w = score.gather(1, torch.topk(value, k, 1).indices)
        if case["renormalize"]:
            w = w / w.sum(1, keepdim=True)
        return [None, case["scale"] * w]
    with torch.enable_grad():
        l.requires_grad_()
        score = torch.softmax(l, 1) if case["score"] == "softmax" else torch.special.expit(l)
        w = score.gather(1, st["ids"].long())
        if case["renormalize"]:
            w = w / w.sum(1, keepdim=True)
        return [torch.autograd.grad(case["scale"] * w, l, st["dweights"].double())[0]]


def _exact_experts(st):
    case, f64 = st["case"], torch.float64
    T, k, E, D, N, act = (case[n] for n in ("T", "k", "E", "D", "N", "act"))

    def weight(name, e, n_rows, n_cols):
        # element by element from the layout's address rule
        wq, scales, zeros = (v.view(E, -1)[e] for v in st[name])
        NB = n_rows // 16
        n = torch.arange(n_rows, device="cuda")[:, None]
        c = torch.arange(n_cols, device="cuda")
        g, kk = c // GROUP, c % GROUP
        j = kk % 8
        slot = j // 2 + 4 * (j % 2)
        lane = 16 * (kk % 32 // 8) + n % 16
        byte = wq[((g * NB + n // 16) * 64 + lane) * 16 + 4 * (kk // 32) + slot // 2]
        q = ((byte >> (4 * (slot % 2)).to(torch.uint8)) & 15).to(f64)
        meta = ((g // 4 * NB + n // 16) * 16 + n % 16) * 4 + g % 4
        return (q - zeros[meta].to(f64)) * scales[meta].to(f64)

    def f(z):
        if act == "relu":
            return torch.where(z > 0, z, 0.0)
        if act == "silu":
            return z * torch.special.expit(z)
        if act == "gelu":
            return z * torch.special.ndtr(z)
        # (1 + tanh a) / 2 = 1 / (1 + exp(-2 a))
        return z * torch.special.expit(math.sqrt(8 / math.pi) * (z + 0.044715 * z ** 3))

    forward = case["op"] == "experts"
    a = (st["X"] if forward else st["dY"]).to(f64)
    s = 1.0 if st["s"] is None else st["s"].to(f64)
    extra = st["residual"] if forward else st["add"]
    y = torch.zeros(T, D, dtype=f64, device="cuda")
    side = [torch.zeros(T, k, N, dtype=f64, device="cuda") for _ in range(2)] if case["train"] else []
    dw = torch.zeros(T, k, dtype=f64, device="cuda")
    for e in range(E):
        token, j = torch.nonzero(st["ids"] == e, as_tuple=True)
        if token.numel() == 0:
            continue
        w = st["weights"][token, j].to(f64)[:, None]
        wd = weight("down", e, D, N)
        if st["s_down"] is not None:
            wd = wd * st["s_down"][e].to(f64)
        wg, wu = weight("gate", e, N, D), weight("up", e, N, D)
        if forward:
            x = a[token] * s
            g, u = torch.matmul(x, wg.T), torch.matmul(x, wu.T)
            if side:
                side[0][token, j], side[1][token, j] = g, u
            y.index_add_(0, token, torch.matmul(f(g) * u, wd.T) * w)
        else:
            g = st["G"][token, j].to(f64)
            u = st["U"][token, j].to(f64)
            dh = torch.matmul(a[token], wd)
            with torch.enable_grad():
                z = g.clone().requires_grad_()
                slope = torch.autograd.grad(f(z).sum(), z)[0]
            dw[token, j] = torch.sum(dh * f(g) * u, 1)
            y.index_add_(0, token, w * (torch.matmul(dh * u * slope, wg) + torch.matmul(dh * f(g), wu)))
    if not forward:
        y = y * s
    if extra is not None:
        y = y + extra.to(f64)
    return [y] + side if forward else [y, dw]


def exact(case, seed):
    st, op = prepare(case, seed), case["op"]
    form = (_exact_norm if op.startswith("norm") else
            _exact_route if op.startswith("route") else _exact_experts)
    return form(st)


def work(case):
    op, T = case["op"], case["T"]
    if op.startswith("norm"):
        D, y, pre = case["D"], case["y"], case["pre"] != "none"
        B = -(-T // case["gate"]) if case["gate"] else 0
        vectors = sum({"none": 0, "rms": 1, "layer": 2}[case[w]] for w in ("post", "pre"))
        if op == "norm":
            return {"bytes": 2.0 * T * D * (1 + 2 * y + pre) + 2 * D * (B + vectors),
                    "flops": 12.0 * T * D}
        # dr, y, dx, dy; dh and r; the gate, the norms' weights, and their fp32 gradients
        weights = (case["post"] != "none") + pre + (case["post"] == "layer" and B > 0)
        return {"bytes": 2.0 * T * D * (4 + 2 * pre) + 2 * D * (B + weights) + 4 * D * (B + vectors),
                "flops": 30.0 * T * D}
    if op.startswith("route"):
        E, k, size = case["E"], case["k"], 4 if case["dtype"] == "fp32" else 2
        if op == "route":
            return {"bytes": float(T * E * size + T * k * 8 + (4 * E if case["bias"] else 0)),
                    "flops": 10.0 * T * E}
        return {"bytes": float(2 * T * E * size + T * k * 8), "flops": 10.0 * T * E}
    E, k, D, N = case["E"], case["k"], case["D"], case["N"]
    slots = T * k * (1 - case["skip"])
    # experts that an even demand reaches, each one's codes, scales and zero points read once
    active = E * (1 - (1 - 1 / E) ** slots) if T > 1 else min(E, slots)
    bytes_ = 3 * active * N * D * (0.5 + 4 / GROUP) + T * k * 8
    bytes_ += 2 * (D + active * N) if case["s"] else 0
    if op == "experts":
        bytes_ += 2 * T * D * (3 if case["residual"] else 2) + (4 * T * k * N if case["train"] else 0)
    else:
        bytes_ += 2 * T * D * (3 if case["residual"] else 2) + 4 * slots * N + 2 * T * k
    return {"bytes": float(bytes_), "flops": 6.0 * slots * N * D}
