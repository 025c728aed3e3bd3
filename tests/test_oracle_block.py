"""The fp64 reference of the expert block: gradients against central differences, and the
routing rules on examples small enough to check by hand."""
import numpy as np
import pytest

from oracle import block


def differences(f, x, d, step=1e-5):
    """Gradient of sum(f(x) * d) by central differences."""
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        a, b = x.copy(), x.copy()
        a[i] += step
        b[i] -= step
        g[i] = ((f(a) - f(b)) * d).sum() / (2 * step)
    return g


@pytest.mark.parametrize("post", block.KINDS)
@pytest.mark.parametrize("pre", block.KINDS)
@pytest.mark.parametrize("gate_rows", [0, 2, 5])
def test_norm_gradients(post, pre, gate_rows):
    rng = np.random.default_rng([5, block.KINDS.index(post), block.KINDS.index(pre), gate_rows])
    T, D, alpha, eps = 5, 6, 0.7, 1e-3
    x, y, dr, dh = (rng.standard_normal((T, D)) for _ in range(4))
    w, b, v, c = (rng.standard_normal(D) for _ in range(4))
    gate = rng.standard_normal((-(-T // gate_rows), D)) if gate_rows else None

    def run(x, y, gate, w, b, v, c):
        r, h = block.norm_block(x, y, (post, w, b, eps), (pre, v, c, eps), gate, gate_rows or 1, alpha)
        return np.concatenate([r, h])
    args = [x, y, gate, w, b, v, c]
    dh_used = dh if pre != "none" else None
    d = np.concatenate([dr, dh if pre != "none" else np.zeros_like(dh)])
    r = block.norm_block(x, y, (post, w, b, eps), ("none",), gate, gate_rows or 1, alpha)[0]
    got = block.norm_block_backward(dr, dh_used, y, r, (post, w, b, eps), (pre, v, c, eps), gate,
                                    gate_rows or 1, alpha)
    for i, name in enumerate(("dx", "dy", "gate", "post_weight", "post_bias", "pre_weight", "pre_bias")):
        if args[i] is None or (post == "none" and name.startswith("post")) or \
                (pre == "none" and name.startswith("pre")):
            assert got[name] is None or name == "gate"
            continue
        ref = differences(lambda t: run(*args[:i], t, *args[i + 1:]), args[i], d)
        assert np.allclose(got[name], ref, rtol=1e-6, atol=1e-7), name


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [False, True])
def test_route_gradients(score, renormalize):
    rng = np.random.default_rng(7)
    T, E, k = 4, 9, 3
    logits, dw = rng.standard_normal((T, E)), rng.standard_normal((T, k))
    ids, w = block.route(logits, k, score, renormalize=renormalize, scale=1.5)

    def weights(l):
        s = np.take_along_axis(block.scores(l, score), ids.astype(int), 1)
        return 1.5 * (s / s.sum(1, keepdims=True) if renormalize else s)
    assert np.allclose(weights(logits), w, rtol=1e-12)
    got = block.route_backward(dw, logits, ids, score, renormalize, 1.5)
    assert np.allclose(got, differences(weights, logits, dw), rtol=1e-6, atol=1e-8)


def test_route_rules():
    inf, nan = np.inf, np.nan
    l = np.array([[0, 2, 1, 2, -1, 0], [-inf, -inf, 1, nan, -inf, -inf], [-inf] * 6,
                  [inf, 0, inf, 1, 0, 0], [1, 1, 1, 1, 1, 1]])
    ids, w = block.route(l, 2)
    assert ids.tolist() == [[1, 3], [2, -1], [-1, -1], [0, 2], [0, 1]]
    assert np.allclose(w, [[0.5, 0.5], [1, 0], [0, 0], [0.5, 0.5], [0.5, 0.5]])
    # a bias cannot bring a masked expert back, and moves the choice but not the weights
    bias = np.array([9.0, 0, 0, 9, 9, 9])
    ids, w = block.route(l[1:2], 2, bias=bias, renormalize=False)
    assert ids.tolist() == [[2, -1]] and np.allclose(w, [[1, 0]])
    ids, w = block.route(l[:1], 2, bias=np.array([0, 0, 0, 0, 9.0, 0]), renormalize=False)
    assert ids.tolist() == [[4, 1]] and np.allclose(w, block.scores(l[:1], "softmax")[:, [4, 1]])
    # groups {0,1} {2,3} {4,5}: sums of the two best 2, 3, -1 in the logits' order
    ids, _ = block.route(l[:1], 2, groups=3, topk_groups=1)
    assert ids.tolist() == [[3, 2]]
    # scores that underflow still have a ratio
    _, w = block.route(np.array([[-900.0, -901.0, -2000.0]]), 2, "sigmoid")
    assert np.allclose(w, [[1 / (1 + np.exp(-1)), 1 / (1 + np.exp(1))]])


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_experts_gradients(act):
    rng = np.random.default_rng(11)
    T, E, k, D, N = 3, 4, 2, 5, 6
    X, dY, R = (rng.standard_normal((T, D)) for _ in range(3))
    gate, up = (rng.standard_normal((E, N, D)) for _ in range(2))
    down = rng.standard_normal((E, D, N))
    ids = np.array([[0, 3], [3, -1], [7, 1]], np.int32)      # -1 and 7 name no expert
    w = rng.random((T, k))
    s, s_down = rng.random(D) + 0.5, rng.random((E, N)) + 0.5

    def run(X, w):
        return block.experts(X, ids, w, gate, up, down, act, s, s_down, R)[0]
    _, G, U = block.experts(X, ids, w, gate, up, down, act, s, s_down)
    dX, dw = block.experts_backward(dY, ids, w, G, U, gate, up, down, act, s, s_down)
    assert np.allclose(dX, differences(lambda t: run(t, w), X, dY), rtol=1e-6, atol=1e-7)
    assert np.allclose(dw, differences(lambda t: run(X, t), w, dY), rtol=1e-6, atol=1e-7)
    assert dw[1, 1] == 0 and dw[2, 0] == 0
