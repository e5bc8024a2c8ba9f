"""Plain float64 forms of the linear layer, the gated block, their backward passes and gradient clipping.

    linear: pre = X W + b; out = act(pre) + R          gated: out = act(X Wg) * (X Wu)
    clip  : n = sqrt(sum g^2); g * min(1, max_norm / (n + eps))

Weights are in the math layout here ([K, N]).  Everything is numpy float64.
"""
from __future__ import annotations

import math

import numpy as np

_erf = np.vectorize(math.erf, otypes=[np.float64])

NONE, GELU_ERF, GELU_TANH, SILU, RELU = range(5)


def _f(x):
    return np.asarray(x, dtype=np.float64)


def _logistic(x):
    e = np.exp(-np.abs(x))
    return np.where(x >= 0, 1.0 / (1.0 + e), e / (1.0 + e))


def act(kind, x):
    x = _f(x)
    if kind == GELU_ERF:
        return 0.5 * x * (1.0 + _erf(x / math.sqrt(2.0)))
    if kind == GELU_TANH:
        return 0.5 * x * (1.0 + np.tanh(math.sqrt(2.0 / math.pi) * (x + 0.044715 * x ** 3)))
    if kind == SILU:
        return x * _logistic(x)
    if kind == RELU:
        return np.maximum(x, 0.0)
    return x


def act_grad(kind, x):
    x = _f(x)
    if kind == GELU_ERF:
        return 0.5 * (1.0 + _erf(x / math.sqrt(2.0))) + x * np.exp(-0.5 * x * x) / math.sqrt(2.0 * math.pi)
    if kind == GELU_TANH:
        t = np.tanh(math.sqrt(2.0 / math.pi) * (x + 0.044715 * x ** 3))
        return 0.5 * (1.0 + t) + 0.5 * x * (1.0 - t * t) * math.sqrt(2.0 / math.pi) * (1.0 + 3 * 0.044715 * x * x)
    if kind == SILU:
        s = _logistic(x)
        return s * (1.0 + x * (1.0 - s))
    if kind == RELU:
        return (x > 0).astype(np.float64)
    return np.ones_like(x)


def linear(X, W, b=None, R=None, kind=NONE):
    """(out, pre)"""
    pre = _f(X) @ _f(W)
    if b is not None:
        pre = pre + _f(b)
    out = act(kind, pre)
    return (out if R is None else out + _f(R)), pre


def linear_backward(X, W, dOut, pre=None, kind=NONE):
    """dict(dPre, dX, dW, dbias)"""
    d = _f(dOut) if kind == NONE else _f(dOut) * act_grad(kind, pre)
    return dict(dPre=d, dX=d @ _f(W).T, dW=_f(X).T @ d, dbias=d.sum(axis=0))


def gated(X, Wg, Wu, kind=SILU):
    """(out, gate, up)"""
    g, u = _f(X) @ _f(Wg), _f(X) @ _f(Wu)
    return act(kind, g) * u, g, u


def gated_backward(X, Wg, Wu, gate, up, dOut, kind=SILU):
    """dict(dGate, dUp, dX, dWg, dWu)"""
    d, g, u = _f(dOut), _f(gate), _f(up)
    dg, du = d * u * act_grad(kind, g), d * act(kind, g)
    return dict(dGate=dg, dUp=du, dX=dg @ _f(Wg).T + du @ _f(Wu).T, dWg=_f(X).T @ dg, dWu=_f(X).T @ du)


def clip(grads, max_norm, eps=1e-6):
    """(norm, [clipped])"""
    norm = math.sqrt(sum(float((_f(g) ** 2).sum()) for g in grads))
    scale = min(1.0, max_norm / (norm + eps)) if norm == norm else norm
    return norm, [_f(g) * scale for g in grads]
