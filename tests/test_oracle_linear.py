"""Pins of the linear / grouped / SwiGLU oracle: closed forms, sums written
out, and every gradient against central differences of the forward function."""
import math

import numpy as np
import pytest

from oracle import ffn as offn
from oracle import linear as ol


def test_activations_at_known_points():
    z = np.array([0.0, 1.0, -1.0, 40.0, -40.0])
    assert np.allclose(ol.act(z, "silu"), [0, 1 / (1 + math.exp(-1)), -1 / (1 + math.e), 40, -40 * math.exp(-40)], rtol=1e-12)
    # Phi(1) = 0.841344746068543 (tables of the normal distribution)
    assert np.allclose(ol.act(z, "gelu")[:3], [0, 0.841344746068543, 0.841344746068543 - 1], rtol=1e-12)
    assert (ol.act(z, "relu") == [0, 1, 0, 40, 0]).all() and (ol.act_slope(z, "relu") == [0, 1, 0, 1, 0]).all()
    for kind in ("silu", "gelu"):   # act(z) - act(-z) = z, slopes add to one
        assert np.allclose(ol.act(z, kind) - ol.act(-z, kind), z, atol=1e-12)
        assert np.allclose(ol.act_slope(z, kind) + ol.act_slope(-z, kind), 1, atol=1e-12)


@pytest.mark.parametrize("kind", ["none", "silu", "gelu", "relu"])
def test_slopes_are_the_differences(kind):
    z = np.linspace(-6, 6, 241) + 0.013
    h = 1e-5
    d = (ol.act(z + h, kind) - ol.act(z - h, kind)) / (2 * h)
    assert np.abs(ol.act_slope(z, kind) - d).max() < 1e-8


@pytest.mark.parametrize("kind", ol.ACTS)
def test_linear_gradients_are_the_differences(kind):
    rng = np.random.default_rng(3)
    T, K, N = 5, 7, 6
    x, w, b, r, dy = (rng.standard_normal(s) for s in ((T, K), (N, K), (N,), (T, N), (T, N)))
    y, z = ol.linear(x, w, b, kind, r)
    assert np.allclose(z[2, 4], sum(x[2, k] * w[4, k] for k in range(K)) + b[4])
    grads = ol.linear_backward(ol.linear_dz(dy, z, kind), x, w)
    loss = lambda: float((ol.linear(x, w, b, kind, r)[0] * dy).sum())
    h = 1e-6
    for arr, grad in zip((x, w, b), grads):
        for i in np.ndindex(arr.shape):
            keep = arr[i]
            arr[i] = keep + h
            up = loss()
            arr[i] = keep - h
            down = loss()
            arr[i] = keep
            assert abs((up - down) / (2 * h) - grad[i]) < 1e-7


def test_grouped_is_the_masked_sum_and_its_gradients_are_the_differences():
    rng = np.random.default_rng(4)
    n, E, K, N = 9, 4, 5, 3
    off = np.array([1, 3, 3, 8, 8])      # row 0 and row 8 belong to no expert; experts 1 and 3 are empty
    x, w, dy = rng.standard_normal((n, K)), rng.standard_normal((E, N, K)), rng.standard_normal((n, N))
    y = ol.grouped(x, w, off)
    owner = [None, 0, 0, 2, 2, 2, 2, 2, None]
    for r, e in enumerate(owner):
        assert np.isnan(y[r]).all() if e is None else np.allclose(y[r], w[e] @ x[r])
    dx, dw = ol.grouped_backward(dy, x, w, off)
    rows = [r for r, e in enumerate(owner) if e is not None]
    loss = lambda: float((ol.grouped(x, w, off)[rows] * dy[rows]).sum())
    h = 1e-6
    for arr, grad in ((x, dx), (w, dw)):
        for i in np.ndindex(arr.shape):
            if arr is x and owner[i[0]] is None:
                assert np.isnan(grad[i])
                continue
            keep = arr[i]
            arr[i] = keep + h
            up = loss()
            arr[i] = keep - h
            down = loss()
            arr[i] = keep
            assert abs((up - down) / (2 * h) - grad[i]) < 1e-7
    assert (dw[1] == 0).all() and (dw[3] == 0).all()


def test_swiglu_is_the_experts_middle_step():
    rng = np.random.default_rng(5)
    gu, dh = rng.standard_normal((4, 12)) * 2, rng.standard_normal((4, 6))
    h = ol.swiglu(gu)
    assert np.allclose(h, offn.silu(gu[:, :6]) * gu[:, 6:])
    grad, step = ol.swiglu_backward(dh, gu), 1e-6
    for i in np.ndindex(gu.shape):
        keep = gu[i]
        gu[i] = keep + step
        up = float((ol.swiglu(gu) * dh).sum())
        gu[i] = keep - step
        down = float((ol.swiglu(gu) * dh).sum())
        gu[i] = keep
        assert abs((up - down) / (2 * step) - grad[i]) < 1e-7
