"""Pins of the fused layers' oracle: values and gradients against differences, the
transposed layout against the packed one."""
import numpy as np
import pytest

import oracle
from oracle import fused as of


@pytest.mark.parametrize("name", of.ACTS)
def test_act_grad_against_differences(name):
    z = np.linspace(-9.0, 9.0, 3601) + 0.0013      # no point at relu's corner
    h = 1e-5
    d = (of.act(z + h, name) - of.act(z - h, name)) / (2 * h)
    # central differences: h^2 / 6 times the third derivative (below 2) plus 1e-16 * 9 / h
    assert np.abs(d - of.act_grad(z, name)).max() < 2e-10 + 2e-10


def test_act_known_values():
    assert of.act(np.array([0.0, 1.0]), "silu")[1] == pytest.approx(0.7310585786300049, abs=1e-15)
    assert of.act(np.array([1.0]), "gelu")[0] == pytest.approx(0.8413447460685429, abs=1e-15)
    assert of.act(np.array([1.0]), "gelu_tanh")[0] == pytest.approx(0.8411919906082768, abs=1e-12)
    assert of.act_grad(np.array([0.0]), "relu")[0] == 0.0
    for name in of.ACTS[1:]:
        assert of.act(np.array([0.0]), name)[0] == 0.0


def test_layer_gradients_against_differences():
    """Directional derivatives of L = sum(dOut * out) with respect to X and the biases."""
    rng = np.random.default_rng(5)
    M, N, K = 7, 48, 128
    X, Wg, Wu = rng.standard_normal((M, K)), rng.standard_normal((N, K)) * 0.1, rng.standard_normal((N, K)) * 0.1
    bg, bu, dH = rng.standard_normal(N), rng.standard_normal(N), rng.standard_normal((M, N))
    dx, h = rng.standard_normal((M, K)), 1e-6
    for name in ("silu", "gelu", "gelu_tanh"):
        H, G, U = of.gated(X, Wg, Wu, name, bg, bu)
        dG, dU = of.gated_grad(dH, G, U, name)
        dX = of.input_grad([dG, dU], [Wg, Wu])

        def loss(x, b):
            return (dH * of.gated(x, Wg, Wu, name, b, bu)[0]).sum()
        num = (loss(X + h * dx, bg) - loss(X - h * dx, bg)) / (2 * h)
        assert (dX * dx).sum() == pytest.approx(num, rel=1e-6)
        db = rng.standard_normal(N)
        num = (loss(X, bg + h * db) - loss(X, bg - h * db)) / (2 * h)
        assert (dG.sum(0) * db).sum() == pytest.approx(num, rel=1e-6)
        Y, Z = of.linear(X, Wg, bg, name, residual=dH)
        dZ = of.linear_grad(dH, Z, name)
        num = ((dH * of.linear(X + h * dx, Wg, bg, name)[0]).sum()
               - (dH * of.linear(X - h * dx, Wg, bg, name)[0]).sum()) / (2 * h)
        assert (of.input_grad([dZ], [Wg]) * dx).sum() == pytest.approx(num, rel=1e-6)


@pytest.mark.parametrize("N,K", [(16, 128), (128, 256), (272, 384)])
def test_transposed_codes_are_the_packed_layout_of_the_transpose(N, K):
    rng = np.random.default_rng(6)
    ng = -(-N // 128)
    for bits, pack in ((4, oracle.pack_codes), (8, oracle.pack_codes8)):
        q = rng.integers(0, 2 ** bits, (N, K)).astype(np.uint8)
        padded = np.zeros((ng * 128, K), dtype=np.uint8)
        padded[:N] = q
        assert np.array_equal(of.transpose_codes(q, bits), pack(np.ascontiguousarray(padded.T)))


def test_transposed_meta():
    rng = np.random.default_rng(7)
    sc = rng.random((144, 3)).astype(np.float16)
    z = rng.integers(0, 16, (144, 3)).astype(np.float16)
    m = of.transpose_meta(sc, z).reshape(2, 3, 2, 128).astype(np.float64)
    for n, u in ((0, 0), (2, 1), (127, 2), (128, 0), (143, 2)):
        assert m[n // 128, u, 0, n % 128] == sc[n, u]
        assert m[n // 128, u, 1, n % 128] == z[n, u] + (64 if n % 4 >= 2 else 1024)
    assert not m[1, :, 0, 16:].any()                       # rows past N: scale 0
    m8 = of.transpose_meta(sc, z, bits=8).reshape(2, 3, 2, 128).astype(np.float64)
    assert m8[0, 1, 1, 2] == z[2, 1] + 1024
