"""fp64 statements of the training operators around the layer (numpy, CPU):
layer norm, the loss head's cross entropy and its distillation.

Test infrastructure only; shares no code with the GPU path.  Every function
takes fp64 arrays of the inputs exactly as stored.
"""
from __future__ import annotations

import numpy as np


def layer_norm(x, w, b, eps):
    mean = x.mean(axis=-1)
    var = ((x - mean[..., None]) ** 2).mean(axis=-1)
    rstd = 1.0 / np.sqrt(var + eps)
    n = (x - mean[..., None]) * rstd[..., None]
    return n * w + (0.0 if b is None else b), mean, rstd


def layer_norm_backward(dy, x, w, mean, rstd):
    n = (x - mean[..., None]) * rstd[..., None]
    g = dy * w
    dx = rstd[..., None] * (g - g.mean(-1, keepdims=True) - n * (g * n).mean(-1, keepdims=True))
    lead = tuple(range(x.ndim - 1))
    return dx, (dy * n).sum(axis=lead), dy.sum(axis=lead)


def one_hot_targets(labels, V):
    """Target distribution [T, V] and which tokens count."""
    T = len(labels)
    P = np.zeros((T, V))
    on = (labels >= 0) & (labels < V)
    P[np.nonzero(on)[0], labels[on]] = 1.0
    return P, on


def teacher_targets(teacher, ids, V, temperature):
    """The teacher's softmax over its entries in use, laid out over the vocabulary."""
    T, K = ids.shape
    P = np.zeros((T, V))
    on = np.zeros(T, dtype=bool)
    entropy = np.zeros(T)                      # sum p log p over the entries, not over the vocabulary
    for t in range(T):
        use = (ids[t] >= 0) & (ids[t] < V) & ~(teacher[t] == -np.inf)
        if not use.any():
            continue
        on[t] = True
        u = teacher[t][use] / temperature
        p = np.exp(u - u.max())
        p /= p.sum()
        np.add.at(P[t], ids[t][use], p)
        entropy[t] = sum(v * np.log(v) for v in p if v > 0)
    return P, on, entropy


def _log_softmax(z):
    m = z.max(axis=1, keepdims=True)
    lse = m[:, 0] + np.log(np.exp(z - m).sum(axis=1))
    return z - lse[:, None], lse


def head_loss(X, W, P, on, entropy, temperature=1.0):
    """(loss, lse) per token; tokens that do not count have 0 in both, whatever X holds there."""
    T = X.shape[0]
    loss, lse = np.zeros(T), np.zeros(T)
    if on.any():
        logq, l = _log_softmax(X[on] @ W.T / temperature)
        lse[on] = l
        loss[on] = temperature ** 2 * (entropy[on] - (P[on] * logq).sum(axis=1))
    return loss, lse


def head_gradients(dloss, X, W, P, on, temperature=1.0):
    """(dX, dW, |D| |W|, |D|^T |X|): the gradients and the sums of magnitudes that bound their rounding."""
    dX, dW = np.zeros_like(X), np.zeros_like(W)
    aX, aW = np.zeros_like(X), np.zeros_like(W)
    on = on & (dloss != 0.0)
    if on.any():
        logq, _ = _log_softmax(X[on] @ W.T / temperature)
        D = (np.exp(logq) - P[on]) * (temperature * dloss[on])[:, None]
        mag = (np.exp(logq) + P[on]) * np.abs(temperature * dloss[on])[:, None]
        dX[on], dW = D @ W, D.T @ X[on]
        aX[on], aW = mag @ np.abs(W), mag.T @ np.abs(X[on])
    return dX, dW, aX, aW
