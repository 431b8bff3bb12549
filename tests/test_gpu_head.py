"""Softmax cross entropy over a quantised head on the GPU against the float64 oracle."""

import numpy as np
import pytest

import oracle
import w4a16_gemm_amd as w4
from experts_common import U, Layers, dev, f16, floored, half_tol, same, within
from gpu_common import device, note

pytestmark = pytest.mark.gpu

SHAPES = [
    # M, N, vocab, K, bits, group, sym, act, without a target
    (1, 8, 8, 64, 4, 32, False, False, 0.0),
    (1, 8, 1, 64, 4, 64, False, False, 0.0),
    (2, 264, 257, 128, 4, 128, False, False, 0.0),
    (37, 1000, 999, 320, 4, 64, True, False, 0.0),
    (64, 5008, 5001, 192, 4, 64, False, False, 0.3),
    (130, 2056, 2056, 256, 4, 256, False, True, 0.1),
    (300, 12808, 12801, 64, 4, 32, False, False, 0.0),
    (700, 1032, 1030, 512, 4, 128, False, False, 0.5),
    (9, 40, 33, 128, 4, 32, False, False, 1.0),
    (1, 16, 16, 64, 8, 64, False, False, 0.0),
    (33, 1040, 1025, 256, 8, 64, True, False, 0.2),
    (270, 4112, 4100, 128, 8, 128, False, True, 0.1),
    (520, 784, 784, 320, 8, 32, False, False, 0.0),
    (20, 66568, 66567, 64, 4, 64, False, False, 0.0),
    (50, 40016, 40016, 192, 8, 64, False, False, 0.1),
    (65, 2056, 2050, 1536, 4, 128, False, False, 0.0),
]


def case(shape):
    M, N, vocab, K, bits, group, sym, act, none = shape
    note(f"head M={M} N={N} vocab={vocab} K={K} bits={bits} group={group} sym={sym} act={act} without={none}")
    rng = np.random.default_rng([95, M, N, K, bits])
    layer = Layers(1, N, K, bits, group, sym, act, experts=False)
    target = rng.integers(0, vocab, M)
    x = f16(rng, (M, K), 2.0)
    sure = rng.random(M)[:, None] * 8.0 / np.maximum(1e-9, (layer.W[0].astype(np.float64) ** 2).sum(1)[target][:, None])
    x = (x + sure * layer.W[0][target].astype(np.float64)).astype(np.float16)
    target[rng.random(M) < none] = rng.choice([-100, -1, vocab, 2 ** 31 - 1])
    return rng, layer, x, target.astype(np.int32), rng.uniform(0.1, 8.0, M).astype(np.float32)


def logit_tol(x, W):
    """[M]: bound of a logit's error, the largest of the row."""
    return 2 * x.shape[1] * U * (floored(x) @ floored(W).T).max(axis=1)


def loss_tol(x, W, lse):
    """(loss, lse): the logits' error; exponentials to 2^-21 of themselves and their argument's
    rounding; sums of 64 + tiles / 8 steps; the logarithm; the last sums' roundings."""
    tl = logit_tol(x, W)
    spread = (np.abs(x.astype(np.float64)) @ np.abs(W.astype(np.float64)).T).max(axis=1) + 12
    rel = 2.0 ** -21 + 4 * U * spread + (64 + W.shape[0] / 2048) * U
    one = tl + rel + 8 * U * (np.abs(lse) + spread)
    return one + tl, one


def dx_tol(dloss, x, W, target, lse, coeff, ref):
    V = W.shape[0]
    e = (loss_tol(x, W, lse)[1] + logit_tol(x, W))[:, None]
    rows = np.nonzero((target >= 0) & (target < V))[0]
    p = np.abs(coeff)
    p[rows, target[rows]] = 1 + coeff[rows, target[rows]]
    err = 1.01 * e * p                               # exponentials
    c = np.abs(coeff)
    rounding = 2.0 ** -11 * c + 2.0 ** -39           # binary16 of c 2^14, half a subnormal step
    rounding[rows, target[rows]] = 2.0 ** -22 * c[rows, target[rows]] + 2.0 ** -24 * p[rows, target[rows]]
    total = (err + rounding + (2 * V + 64) * U * np.maximum(c, 2.0 ** -28)) @ floored(W)
    total[~np.isin(np.arange(len(x)), rows)] = 0
    d = np.abs(dloss.astype(np.float64))[:, None]
    return d * total * 1.001 + half_tol(np.abs(ref) + d * total)


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_loss(shape):
    M, N, vocab, K = shape[:4]
    rng, layer, x, target, dloss = case(shape)
    got = layer.fn("head_loss")(dev(x), *layer.args, dev(target), vocab=vocab)
    loss, lse, coeff = oracle.head_loss(x, layer.W[0], target, vocab)
    tol = loss_tol(x, layer.W[0][:vocab], lse)
    within("loss", got[0], loss, tol[0])
    within("lse", got[1], lse, tol[1])
    out = ((target < 0) | (target >= vocab))
    assert not got[0].cpu().numpy()[out].any() and not got[1].cpu().numpy()[out].any()
    again = layer.fn("head_loss")(dev(x), *layer.args, dev(target), vocab=vocab)
    assert same(got[0], again[0]) and same(got[1], again[1])


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_gradient(shape):
    M, N, vocab, K = shape[:4]
    rng, layer, x, target, dloss = case(shape)
    loss, lse, coeff = oracle.head_loss(x, layer.W[0], target, vocab)
    run = lambda: layer.fn("head_loss_backward")(dev(dloss), dev(x), *layer.args, dev(target),   # noqa: E731
                                                 dev(lse.astype(np.float32)), vocab=vocab)
    dx = run()
    ref = oracle.head_loss_backward(dloss, x, layer.W[0], target, vocab)
    within("dx", dx, ref, dx_tol(dloss, x, layer.W[0][:vocab], target, lse, coeff, ref))
    assert same(dx, run())
