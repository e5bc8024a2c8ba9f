"""Plain float64 forms of the vocabulary cross entropy, its gradients and the AdamW step.

    z = X W; lse = ln sum e^z; loss = lse - z[target], 0 for ignored targets
    dz = (g + h) e^(z - lse) - [target] g, 0 for ignored targets; dX = dz W^T; dW = X^T dz
    m = b1 m + (1 - b1) g; v = b2 v + (1 - b2) g^2
    p = p - lr (decay p + (m / (1 - b1^t)) / (sqrt(v / (1 - b2^t)) + eps))

Weights are in the math layout here ([K, V]).  Everything is numpy float64.
"""
from __future__ import annotations

import numpy as np

BLOCK = 256


def _f(x):
    return np.asarray(x, dtype=np.float64)


def lse_of(z):
    """ln sum e^z of each row, the formula's value where logits are infinite or NaN."""
    top = np.max(np.where(np.isnan(z), -np.inf, z), axis=1, keepdims=True)
    shift = np.where(np.isfinite(top), top, 0.0)
    with np.errstate(over="ignore", divide="ignore", invalid="ignore"):
        return (shift + np.log(np.exp(z - shift).sum(axis=1, keepdims=True)))[:, 0]


def cross_entropy(X, W, targets, ignore=-100, begin=0):
    """dict(z, lse, loss, stats): of the piece that holds the ids from `begin` on."""
    with np.errstate(invalid="ignore", over="ignore"):
        z = _f(X) @ _f(W)
    V = z.shape[1]
    t = np.asarray(targets) - begin
    held = (t >= 0) & (t < V)
    logit = np.where(held, z[np.arange(len(t)), np.clip(t, 0, V - 1)], -np.inf)
    lse = lse_of(z)
    top = np.max(np.where(np.isnan(z), -np.inf, z), axis=1)
    with np.errstate(invalid="ignore", over="ignore"):
        total = np.exp(z - np.where(np.isfinite(top), top, 0.0)[:, None]).sum(axis=1)
        loss = np.where(np.asarray(targets) == ignore, 0.0, lse - logit)
    return dict(z=z, lse=lse, loss=loss, stats=np.stack([top, total, logit]))


def cross_entropy_backward(X, W, targets, lse, g=1.0, h=0.0, ignore=-100, begin=0):
    """dict(q, dz, dX, dW); q = e^(z - lse)"""
    X, W, t = _f(X), _f(W), np.asarray(targets)
    M, V = X.shape[0], W.shape[1]
    on = t != ignore
    X = np.where(on[:, None], X, 0.0)      # an ignored row is no part of anything
    g, h = np.broadcast_to(_f(g), (M,)) * on, np.where(on, np.broadcast_to(_f(h), (M,)), 0.0)
    q = np.exp(X @ W - np.where(on, _f(lse), 0.0)[:, None]) * on[:, None]
    dz = (g + h)[:, None] * q
    held = (t >= begin) & (t < begin + V)
    dz[np.arange(M)[held], (t - begin)[held]] -= g[held]
    return dict(q=q, dz=dz, dX=dz @ W.T, dW=X.T @ dz)


def codes(x, top):
    """(where x lies between codes, scales): x = scale sign(q) (q / top)^2."""
    x = _f(x).ravel()
    pad = -len(x) % BLOCK
    rows = np.abs(np.concatenate([x, np.zeros(pad)])).reshape(-1, BLOCK)
    scale = rows.max(axis=1)
    q = top * np.sqrt(rows / np.where(scale > 0, scale, 1.0)[:, None])
    return q.ravel()[:len(x)] * np.sign(x), scale


def values(q, scale, top):
    q = _f(q).ravel()
    s = np.repeat(_f(scale), BLOCK)[:len(q)]
    return np.sign(q) * (q / top) ** 2 * s


def adamw(p, g, m, v, *, step, lr, beta1=0.9, beta2=0.999, eps=1e-8, decay=0.0, factor=1.0):
    """(param, m, v)"""
    p, g, m, v = _f(p), _f(g) * factor, _f(m), _f(v)
    m = beta1 * m + (1 - beta1) * g
    v = beta2 * v + (1 - beta2) * g * g
    move = (m / (1 - beta1 ** step)) / (np.sqrt(v / (1 - beta2 ** step)) + eps)
    return p - lr * (decay * p + move), m, v
