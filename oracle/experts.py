"""Mixtures of experts of the quantised layer and the softmax cross entropy over a quantised
head, in float64.

The weights enter as binary16((q - Z) S) (``dequant_fp16``), [E][N][K] or [N][K]; an index or a
target outside its range is a slot without an expert, or a row without a target.
"""

from __future__ import annotations

import numpy as np


def route(logits, top_k: int, renormalise: bool = True):
    """(index int32 [M][top_k], weights float64 [M][top_k], p float64 [M][E])."""
    l = np.asarray(logits, np.float64)
    M, E = l.shape
    index = np.full((M, top_k), -1, np.int32)
    weights = np.zeros((M, top_k))
    p = np.zeros((M, E))
    for m in range(M):
        choice = [j for j in range(E) if l[m, j] > -np.inf]
        if choice:
            top = max(l[m, j] for j in choice)
            with np.errstate(invalid="ignore"):
                e = np.exp(l[m] - top)
            p[m] = e / e.sum()
        choice.sort(key=lambda j: (-l[m, j], j))
        for t, j in enumerate(choice[:top_k]):
            index[m, t] = j
            weights[m, t] = p[m, j]
        if renormalise and choice:
            weights[m] /= weights[m].sum()
    return index, weights, p


def route_backward(dweights, logits, index, weights, renormalise: bool = True):
    """dlogits float64 [M][E], by the chain rule through the softmax's Jacobian."""
    dw = np.asarray(dweights, np.float64)
    w = np.asarray(weights, np.float64)
    M, E = np.asarray(logits).shape
    p = route(logits, 1)[2]
    out = np.zeros((M, E))
    for m in range(M):
        ok = [t for t in range(dw.shape[1]) if 0 <= index[m][t] < E]
        if renormalise:
            for t in ok:
                for u in ok:
                    out[m, index[m][t]] += dw[m, u] * w[m, u] * ((t == u) - w[m, t])
        else:
            for t in ok:
                jac = -p[m] * w[m, t]
                jac[index[m][t]] += w[m, t]
                out[m] += dw[m, t] * jac
    return out


def experts_gemm(x, weights, index):
    """y float64 [M][T][N] for index [M][T]."""
    x = np.asarray(x, np.float64)
    y = np.zeros(index.shape + (weights.shape[1],))
    for e in range(weights.shape[0]):
        m, t = np.nonzero(index == e)
        y[m, t] = x[m] @ np.asarray(weights[e], np.float64).T
    return y


def experts_backward(dy, weights, index, dx0=None):
    """dx float64 [M][K]."""
    dy = np.asarray(dy, np.float64)
    dx = np.zeros((dy.shape[0], weights.shape[2])) if dx0 is None else np.asarray(dx0, np.float64).copy()
    for e in range(weights.shape[0]):
        m, t = np.nonzero(index == e)
        np.add.at(dx, m, dy[m, t] @ np.asarray(weights[e], np.float64))
    return dx


def experts_combine(y, weights):
    return (np.asarray(weights, np.float64)[:, :, None] * np.asarray(y, np.float64)).sum(axis=1)


def experts_combine_backward(dout, y, weights):
    """(dy float64 [M][T][N], dweights float64 [M][T])."""
    d = np.asarray(dout, np.float64)[:, None, :]
    return np.asarray(weights, np.float64)[:, :, None] * d, (np.asarray(y, np.float64) * d).sum(axis=2)


def head_loss(x, weights, target, vocab=None):
    """(loss, lse, coefficients p - onehot [M][vocab]) in float64, zeros for rows without a target."""
    x = np.asarray(x, np.float64)
    w = np.asarray(weights, np.float64)[:vocab]
    M, V = x.shape[0], w.shape[0]
    loss, lse, coeff = np.zeros(M), np.zeros(M), np.zeros((M, V))
    for m in range(M):
        t = int(target[m])
        if not 0 <= t < V:
            continue
        l = w @ x[m]
        top = l.max()
        lse[m] = top + np.log(np.exp(l - top).sum())
        loss[m] = lse[m] - l[t]
        coeff[m] = np.exp(l - lse[m])
        coeff[m, t] -= 1.0
    return loss, lse, coeff


def head_loss_backward(dloss, x, weights, target, vocab=None):
    """dx float64 [M][K]."""
    coeff = head_loss(x, weights, target, vocab)[2]
    rows = coeff.any(axis=1)
    dx = np.zeros(np.asarray(x).shape)
    dx[rows] = np.asarray(dloss, np.float64)[rows, None] * (coeff[rows] @ np.asarray(weights, np.float64)[:vocab])
    return dx
