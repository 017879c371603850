"""CPU oracle of the layer norm and the low-rank adapters, in 64 bits -- TEST INFRASTRUCTURE.

The definitions of include/qlin.h written out with numpy, one row (norm) or
one adapter (adapters) at a time; no code is shared with the CUDA path.
Inputs are CPU torch tensors or numpy arrays of any floating type, outputs
numpy float64, unrounded. Pinned by tests/test_oracle_norm_lora.py against
central differences, closed forms and torch's autograd.
"""
from __future__ import annotations

import numpy as np


def _f64(x) -> np.ndarray:
    return x.double().numpy() if hasattr(x, "double") else np.asarray(x, dtype=np.float64)


def layer_norm_forward(X, gamma=None, beta=None, eps: float = 1e-6):
    """(y, mean, rstd)"""
    x = _f64(X)
    mean = x.mean(axis=1)
    rstd = 1.0 / np.sqrt(((x - mean[:, None]) ** 2).mean(axis=1) + eps)
    y = (x - mean[:, None]) * rstd[:, None]
    if gamma is not None:
        y = y * _f64(gamma)
    if beta is not None:
        y = y + _f64(beta)
    return y, mean, rstd


def layer_norm_backward(dY, X, mean, rstd, gamma=None):
    """(dX, dgamma, dbeta) at the given mean and rstd"""
    x, dy, mean, rstd = _f64(X), _f64(dY), _f64(mean), _f64(rstd)
    xh = (x - mean[:, None]) * rstd[:, None]
    d = dy if gamma is None else dy * _f64(gamma)
    m1, m2 = d.mean(axis=1, keepdims=True), (d * xh).mean(axis=1, keepdims=True)
    return rstd[:, None] * (d - m1 - xh * m2), (dy * xh).sum(axis=0), dy.sum(axis=0)


def lora_forward(X, A, B, scale, idx, Y):
    """(Y + update, H); H is NaN in rows without an adapter"""
    x, a, b, s, y = _f64(X), _f64(A), _f64(B), _f64(scale), _f64(Y).copy()
    h = np.full((x.shape[0], a.shape[1]), np.nan)
    for m, l in enumerate(np.asarray(idx)):
        if 0 <= l < a.shape[0]:
            h[m] = a[l] @ x[m]
            y[m] += s[l] * (b[l] @ h[m])
    return y, h


def lora_backward(dY, X, A, B, scale, idx, H, dX):
    """(dX + update, dA, dB, dH); dH is NaN in rows without an adapter"""
    dy, x, a, b, s, h, dx = _f64(dY), _f64(X), _f64(A), _f64(B), _f64(scale), _f64(H), _f64(dX).copy()
    dA, dB = np.zeros(a.shape), np.zeros(b.shape)
    dh = np.full(h.shape, np.nan)
    for m, l in enumerate(np.asarray(idx)):
        if 0 <= l < a.shape[0]:
            dh[m] = s[l] * (dy[m] @ b[l])
            dx[m] += dh[m] @ a[l]
            dA[l] += np.outer(dh[m], x[m])
            dB[l] += s[l] * np.outer(dy[m], h[m])
    return dx, dA, dB, dh
