"""fp64 reference of the fused linear layers and their gradients.

The product is the definition of ``matmul``; around it a layer adds a bias, an
activation and a residual (``linear``), or multiplies the activated gate product by
the up product (``gated``).  The gradients are those of these formulas with the
weights held fixed.  The transposed copy that the backward product reads is restated
element by element from its address rule.
TEST INFRASTRUCTURE: see the package docstring for who may import this.
"""
from __future__ import annotations

import math

import numpy as np
from scipy.special import erfc, expit

_GROUP = 128
_C = math.sqrt(2.0 / math.pi)
ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")


def act(z: np.ndarray, name: str) -> np.ndarray:
    z = np.asarray(z, dtype=np.float64)
    if name == "none":
        return z
    if name == "relu":
        return np.where(z > 0, z, 0.0)
    if name == "silu":
        return z * expit(z)
    if name == "gelu":
        return 0.5 * z * erfc(-z / math.sqrt(2.0))
    if name == "gelu_tanh":
        # (1 + tanh u) / 2 = 1 / (1 + exp(-2 u))
        return z * expit(2.0 * _C * (z + 0.044715 * z ** 3))
    raise ValueError(name)


def act_grad(z: np.ndarray, name: str) -> np.ndarray:
    z = np.asarray(z, dtype=np.float64)
    if name == "none":
        return np.ones_like(z)
    if name == "relu":
        return np.where(z > 0, 1.0, 0.0)
    if name == "silu":
        sg = expit(z)
        return sg + z * sg * expit(-z)
    if name == "gelu":
        return 0.5 * erfc(-z / math.sqrt(2.0)) + z * np.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    if name == "gelu_tanh":
        u2 = 2.0 * _C * (z + 0.044715 * z ** 3)
        sg = expit(u2)
        return sg + z * sg * expit(-u2) * 2.0 * _C * (1.0 + 3.0 * 0.044715 * z * z)
    raise ValueError(name)


def linear(X, W, bias=None, act_name="none", residual=None):
    """(Y, Z): Z = X . W^T + bias, Y = residual + act(Z), with W = W_hat [N][K] in fp64."""
    Z = np.asarray(X, np.float64) @ W.T
    if bias is not None:
        Z = Z + np.asarray(bias, np.float64)
    Y = act(Z, act_name)
    return (Y if residual is None else Y + np.asarray(residual, np.float64)), Z


def gated(X, Wg, Wu, act_name="silu", bias_gate=None, bias_up=None):
    """(H, G, U): H = act(G) * U."""
    _, G = linear(X, Wg, bias_gate)
    _, U = linear(X, Wu, bias_up)
    return act(G, act_name) * U, G, U


def linear_grad(dY, Z, act_name="none"):
    """dZ = dY * act'(Z)."""
    dY = np.asarray(dY, np.float64)
    return dY if act_name == "none" else dY * act_grad(Z, act_name)


def gated_grad(dH, G, U, act_name="silu"):
    """(dG, dU)."""
    dH, G, U = (np.asarray(a, np.float64) for a in (dH, G, U))
    return dH * U * act_grad(G, act_name), dH * act(G, act_name)


def input_grad(dZs, Ws, add=None):
    """dX = add + sum of dZ . W_hat."""
    dX = sum(np.asarray(d, np.float64) @ W for d, W in zip(dZs, Ws))
    return dX if add is None else dX + np.asarray(add, np.float64)


def transpose_codes(q: np.ndarray, bits: int = 4) -> np.ndarray:
    """The transposed copy's code bytes of q [N][K]: 16 x 128 tiles of q^T, the output
    rows padded with code 0 to a multiple of 128."""
    N, K = q.shape
    ng = -(-N // _GROUP)
    size = 2048 if bits == 8 else 1024
    out = np.zeros(ng * (K // 16) * size, dtype=np.uint8)
    n, k = np.meshgrid(np.arange(N), np.arange(K), indexing="ij")
    g, j = n // _GROUP, n % _GROUP
    t, c, e = j // 32, j % 32 // 8, j % 8
    base = (g * (K // 16) + k // 16) * size
    lane = 16 * c + k % 16
    if bits == 8:
        out[base + 32 * lane + 8 * t + e] = q
        return out
    slot = e // 2 + 4 * (e % 2)
    np.bitwise_or.at(out, base + 16 * lane + 4 * t + slot // 2,
                     (q.astype(np.uint8) << (4 * (slot % 2)).astype(np.uint8)))
    return out


def transpose_meta(scales: np.ndarray, zeros: np.ndarray, bits: int = 4) -> np.ndarray:
    """The transposed copy's metadata (fp16 elements) of scales, zeros [N][K/128]."""
    N, G = scales.shape
    ng = -(-N // _GROUP)
    out = np.zeros((ng, G, 2, _GROUP), dtype=np.float16)
    bias = np.full(_GROUP, 1024.0)
    if bits == 4:
        bias[np.arange(_GROUP) % 4 >= 2] = 64.0
    out[:, :, 1, :] = bias.astype(np.float16)
    for n in range(N):
        out[n // _GROUP, :, 0, n % _GROUP] = scales[n]
        out[n // _GROUP, :, 1, n % _GROUP] = zeros[n].astype(np.float64) + bias[n % _GROUP]
    return out.reshape(-1)
