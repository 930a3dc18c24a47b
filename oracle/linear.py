"""Linear and grouped linear products, SwiGLU rows, and their gradients, in fp64.

    linear     z = x W^T + b,  y = act(z) + r;   dz = dy act'(z),  dx = dz W,
               dW = dz^T x,  db = sum_t dz[t]
    grouped    the product of rows offsets[e] .. offsets[e + 1] with W[e]
    swiglu     h = silu(g) u  ("Llama 开源模型系列" (docs.ifdog.com), "SwiGLU：门控激活的数学")

Readings: GELU is the exact form z Phi(z); ReLU's derivative at 0 is 0.
Inputs are numpy arrays (any float type); nothing here rounds.
"""
from __future__ import annotations

import math

import numpy as np

ACTS = ("none", "relu", "silu", "gelu")
_erfc = np.vectorize(math.erfc, otypes=[np.float64])


def sigmoid(z: np.ndarray) -> np.ndarray:
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-z))


def act(z: np.ndarray, kind: str) -> np.ndarray:
    if kind == "relu":
        return np.maximum(z, 0.0)
    if kind == "silu":
        return z * sigmoid(z)
    if kind == "gelu":
        return z * 0.5 * _erfc(-z / math.sqrt(2.0)) if z.size else z
    return z


def act_slope(z: np.ndarray, kind: str) -> np.ndarray:
    if kind == "relu":
        return (z > 0).astype(np.float64)
    if kind == "silu":
        s = sigmoid(z)
        return s * (1.0 + z * (1.0 - s))
    if kind == "gelu":
        cdf = 0.5 * _erfc(-z / math.sqrt(2.0)) if z.size else z
        return cdf + z * np.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    return np.ones_like(z)


def linear(x, w, bias=None, kind="none", residual=None):
    """(y, z)"""
    z = x.astype(np.float64) @ w.astype(np.float64).T
    if bias is not None:
        z = z + bias.astype(np.float64)
    y = act(z, kind)
    if residual is not None:
        y = y + residual.astype(np.float64)
    return y, z


def linear_dz(dy, z, kind):
    dz = dy.astype(np.float64)
    return dz if kind == "none" else dz * act_slope(z.astype(np.float64), kind)


def linear_backward(dz, x, w):
    """(dx, dw, db) from dz"""
    dz = dz.astype(np.float64)
    return dz @ w.astype(np.float64), dz.T @ x.astype(np.float64), dz.sum(0)


def grouped(x, w, offsets):
    """y; rows of no expert are NaN"""
    y = np.full((x.shape[0], w.shape[1]), np.nan)
    for e in range(w.shape[0]):
        s = slice(int(offsets[e]), int(offsets[e + 1]))
        y[s] = x[s].astype(np.float64) @ w[e].astype(np.float64).T
    return y


def grouped_backward(dy, x, w, offsets):
    """(dx, dw); dx's rows of no expert are NaN"""
    dx = np.full(x.shape, np.nan)
    dw = np.zeros(w.shape)
    for e in range(w.shape[0]):
        s = slice(int(offsets[e]), int(offsets[e + 1]))
        dx[s] = dy[s].astype(np.float64) @ w[e].astype(np.float64)
        dw[e] = dy[s].astype(np.float64).T @ x[s].astype(np.float64)
    return dx, dw


def swiglu(gu):
    g, u = np.split(gu.astype(np.float64), 2, axis=1)
    return act(g, "silu") * u


def swiglu_backward(dh, gu):
    g, u = np.split(gu.astype(np.float64), 2, axis=1)
    dh = dh.astype(np.float64)
    return np.concatenate([dh * u * act_slope(g, "silu"), dh * act(g, "silu")], axis=1)
