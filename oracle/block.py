"""Reference of the expert feed-forward block in fp64 NumPy: the norms before and after a block
with its gate and residual scale, the routing to experts, and the experts' gated feed-forward
blocks, with their backward passes written from the formulas.  No code of the library.
TEST INFRASTRUCTURE: see the package docstring for who may import this.
"""
import numpy as np

from .fused import act, act_grad

KINDS = ("none", "rms", "layer")


# ---- norms ---------------------------------------------------------------------------------

def normalized(v, kind, eps):
    """(normalised rows, 1 / their deviation)."""
    if kind == "layer":
        v = v - v.mean(1, keepdims=True)
    inv = 1.0 / np.sqrt((v * v).mean(1, keepdims=True) + eps)
    return v * inv, inv


def norm(v, kind, weight=None, bias=None, eps=1e-6):
    if kind == "none":
        return v
    n = normalized(v, kind, eps)[0]
    if weight is not None:
        n = n * weight
    return n if bias is None else n + bias


def gate_of(gate, gate_rows, T):
    return 1.0 if gate is None else gate[np.arange(T) // gate_rows]


def norm_block(x, y=None, post=("none",), pre=("none",), gate=None, gate_rows=1, alpha=1.0):
    """(r, h); post and pre: (kind, weight, bias, eps) as for norm()."""
    r = alpha * x
    if y is not None:
        r = r + gate_of(gate, gate_rows, len(x)) * norm(y, *post)
    return r, norm(r, *pre)


def _norm_backward(d, v, kind, weight=None, bias=None, eps=1e-6):
    """(gradient of v, of the weight, of the bias) from that of the norm's output."""
    n, inv = normalized(v, kind, eps)
    dw, db = (d * n).sum(0), d.sum(0)
    if weight is not None:
        d = d * weight
    d = d - n * (d * n).mean(1, keepdims=True) - (d.mean(1, keepdims=True) if kind == "layer" else 0.0)
    return d * inv, dw, db


def norm_block_backward(dr, dh, y=None, r=None, post=("none",), pre=("none",), gate=None, gate_rows=1,
                        alpha=1.0):
    """Dict of dx, dy, gate, post_weight, post_bias, pre_weight, pre_bias."""
    out = dict.fromkeys(("dx", "dy", "gate", "post_weight", "post_bias", "pre_weight", "pre_bias"))
    R = 0.0 if dr is None else dr
    if pre[0] != "none":
        d, out["pre_weight"], out["pre_bias"] = _norm_backward(dh, r, *pre)
        R = R + d
    out["dx"] = alpha * R
    if y is not None:
        g = gate_of(gate, gate_rows, len(R))
        if gate is not None:
            p = R * norm(y, *post)
            out["gate"] = np.stack([p[b * gate_rows:(b + 1) * gate_rows].sum(0) for b in range(len(gate))])
        p = R * g
        if post[0] == "none":
            out["dy"] = p
        else:
            out["dy"], out["post_weight"], out["post_bias"] = _norm_backward(p, y, *post)
    return out


# ---- routing ---------------------------------------------------------------------------------

def _clean(logits):
    """-inf where an expert may not be chosen; +inf as the largest fp32 value."""
    l = np.where(np.isnan(logits), -np.inf, logits.astype(np.float64))
    return np.minimum(l, float(np.finfo(np.float32).max))


def scores(logits, score):
    l = _clean(logits)
    with np.errstate(over="ignore", invalid="ignore"):
        if score == "sigmoid":
            return np.where(l == -np.inf, 0.0, 1.0 / (1.0 + np.exp(-l)))
        top = l.max(1, keepdims=True)
        e = np.where(l == -np.inf, 0.0, np.exp(l - top))
        s = e.sum(1, keepdims=True)
    return np.divide(e, s, out=np.zeros_like(e), where=s > 0)


def route(logits, k, score="softmax", bias=None, groups=1, topk_groups=1, renormalize=True, scale=1.0):
    """(ids, weights): token by token, by sorting."""
    T, E = logits.shape
    l, s = _clean(logits), scores(logits, score)
    ids, weights = np.full((T, k), -1, np.int32), np.zeros((T, k))
    for t in range(T):
        may = [e for e in range(E) if l[t, e] != -np.inf]
        value = s[t] if bias is None else s[t] + bias.astype(np.float64)
        # without a bias the logits order the scores, also where scores round together
        order = l[t] if bias is None else value
        if topk_groups < groups:
            size = E // groups
            best = []
            for g in range(groups):
                inside = sorted((value[e] for e in may if e // size == g), reverse=True)[:2]
                if inside:
                    best.append((-sum(inside), g))
            kept = {g for _, g in sorted(best)[:topk_groups]}
            may = [e for e in may if e // size in kept]
        chosen = sorted(may, key=lambda e: (-order[e], e))[:k]
        if not chosen:
            continue
        w = s[t, chosen]
        if renormalize:
            w = shares(l[t, chosen], score)
        ids[t, :len(chosen)], weights[t, :len(chosen)] = chosen, scale * w
    return ids, weights


def shares(l, score):
    """Scores over their sum, from logits, where the scores themselves may underflow."""
    if score == "sigmoid":  # log sigmoid
        l = np.minimum(l, 0.0) - np.log1p(np.exp(-np.abs(l)))
    e = np.exp(l - l.max())
    return e / e.sum()


def route_backward(dweights, logits, ids, score="softmax", renormalize=True, scale=1.0, **_):
    T, E = logits.shape
    l, s = _clean(logits), scores(logits, score)
    d = np.zeros((T, E))
    for t in range(T):
        slots = [j for j, e in enumerate(ids[t]) if 0 <= e < E and l[t, e] != -np.inf]
        if not slots:
            continue
        e, g = ids[t, slots], scale * dweights[t, slots]
        if renormalize:
            q = shares(l[t, e], score)
            g = q * (g - (q * g).sum())
            if score == "sigmoid":
                with np.errstate(over="ignore"):  # (a score of 1: no gradient)
                    g = g / (1.0 + np.exp(l[t, e]))
            np.add.at(d[t], e, g)
        elif score == "sigmoid":
            np.add.at(d[t], e, g * s[t, e] * (1.0 - s[t, e]))
        else:
            full = np.zeros(E)
            np.add.at(full, e, g)
            d[t] = s[t] * (full - (s[t] * full).sum())
    return d


# ---- experts ---------------------------------------------------------------------------------

def experts(X, ids, weights, gate, up, down, act_name="silu", s=None, s_down=None, residual=None):
    """(Y, G, U); gate, up [E][N][D] and down [E][D][N] dequantized without s, G and U [T][k][N]
    (0 in slots that name no expert)."""
    T, k = ids.shape
    E, N = gate.shape[:2]
    Y = np.zeros_like(X, dtype=np.float64) if residual is None else residual.copy()
    G, U = np.zeros((T, k, N)), np.zeros((T, k, N))
    xs = X if s is None else X * s
    for e in range(E):
        t, j = np.nonzero(ids == e)
        if not len(t):
            continue
        g, u = xs[t] @ gate[e].T, xs[t] @ up[e].T
        G[t, j], U[t, j] = g, u
        h = act(g, act_name) * u
        if s_down is not None:
            h = h * s_down[e]
        np.add.at(Y, t, weights[t, j][:, None] * (h @ down[e].T))
    return Y, G, U


def experts_backward(dY, ids, weights, G, U, gate, up, down, act_name="silu", s=None, s_down=None, add=None):
    """(dX, dweights)."""
    T, k = ids.shape
    E = gate.shape[0]
    dX, dw = np.zeros((T, gate.shape[2])), np.zeros((T, k))
    for e in range(E):
        t, j = np.nonzero(ids == e)
        if not len(t):
            continue
        dh = dY[t] @ down[e]
        if s_down is not None:
            dh = dh * s_down[e]
        g, u = G[t, j], U[t, j]
        a = act(g, act_name)
        dw[t, j] = (dh * a * u).sum(1)
        dh = dh * weights[t, j][:, None]
        np.add.at(dX, t, (dh * u * act_grad(g, act_name)) @ gate[e] + (dh * a) @ up[e])
    if s is not None:
        dX = dX * s
    return dX if add is None else dX + add, dw
