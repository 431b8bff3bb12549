"""Low-rank adapters beside the layer, their gradients, and activations kept in 8 bits, in
float64.

Forward: out[m] = y[m] + s_i B_i (A_i x[m]) with i = index[m]; rows whose index lies outside
[0, L) are y[m].  The gradients are those of sum(dy * out) with respect to x (added to
dx0), A and B.  The 8-bit scheme is the symmetric round-to-nearest quantiser
("LLM Quantization: INT8, GPTQ, and AWQ Explained", What quantization actually does) on
rows of activations.
"""

from __future__ import annotations

import numpy as np

from .quant import fp16_ceil, round_half_even

ACT_MAX_SCALE = 515.5     # largest binary16 S with a finite binary16(127 S)


def _rows(index, M: int, L: int):
    owner = np.zeros(M, np.int64) if index is None else np.asarray(index, np.int64)
    return [np.nonzero(owner == i)[0] for i in range(L)]


def _scaling(scaling, L: int):
    return np.ones(L) if scaling is None else np.asarray(scaling, np.float64)


def lora_forward(y, x, a, b, index=None, scaling=None):
    """(out float64 [M][N], h float64 [M][R]), unrounded."""
    y, x, a, b = (np.asarray(t, np.float64) for t in (y, x, a, b))
    s = _scaling(scaling, a.shape[0])
    out = y.copy()
    h = np.zeros((x.shape[0], a.shape[1]))
    for i, rows in enumerate(_rows(index, x.shape[0], a.shape[0])):
        h[rows] = x[rows] @ a[i].T
        out[rows] += s[i] * (h[rows] @ b[i].T)
    return out, h


def lora_backward(dy, x, a, b, h, index=None, scaling=None, dx0=None):
    """(dx float64 [M][K], da [L][R][K], db [L][N][R]), unrounded."""
    dy, x, a, b, h = (np.asarray(t, np.float64) for t in (dy, x, a, b, h))
    s = _scaling(scaling, a.shape[0])
    dx = np.zeros(x.shape) if dx0 is None else np.asarray(dx0, np.float64).copy()
    da, db = np.zeros(a.shape), np.zeros(b.shape)
    for i, rows in enumerate(_rows(index, x.shape[0], a.shape[0])):
        g = dy[rows] @ b[i]
        dx[rows] += s[i] * (g @ a[i])
        da[i] = s[i] * (g.T @ x[rows])
        db[i] = s[i] * (dy[rows].T @ h[rows])
    return dx, da, db


def act_quantize(x, group_size: int):
    """binary16 x [M][K] -> (codes uint8 [M][K], scales binary16 [M][K / group_size])."""
    x = np.asarray(x, np.float16).astype(np.float64)
    M, K = x.shape
    g = x.reshape(M, K // group_size, group_size)
    finite = np.isfinite(g).all(axis=2)
    g = np.where(finite[..., None], g, 0.0)
    top = np.abs(g).max(axis=2)
    s = np.where(top == 0, 1.0, np.minimum(fp16_ceil(top / 127.0).astype(np.float64), ACT_MAX_SCALE))
    q = np.clip(round_half_even(g / s[..., None]), -127, 127)
    scales = np.where(finite, s, np.nan).astype(np.float16)
    return (q + 128).astype(np.uint8).reshape(M, K), scales


def act_values(codes, scales, group_size: int) -> np.ndarray:
    """binary16((codes - 128) * scale) as [M][K]."""
    s = np.repeat(np.asarray(scales, np.float16).astype(np.float64), group_size, axis=1)
    return ((np.asarray(codes, np.float64) - 128.0) * s).astype(np.float16)
