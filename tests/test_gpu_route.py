"""Routing and the weighted sum of experts' outputs on the GPU against the float64 oracle."""

import numpy as np
import pytest

import oracle
import w4a16_gemm_amd as w4
from experts_common import U, dev, f16, half_tol, same, within
from gpu_common import device, note

pytestmark = pytest.mark.gpu

SIZES = [(1, 1, 1), (1, 2, 2), (3, 7, 4), (17, 8, 2), (65, 16, 16), (33, 17, 3), (100, 64, 8), (257, 65, 1), (40, 128, 8),
         (30, 129, 10), (19, 256, 64), (21, 257, 8), (9, 512, 512), (4000, 60, 4)]


def logits_of(rng, M, E, kind, how):
    l = rng.standard_normal((M, E)) * 2
    if how == "ties":
        l = np.round(l)
        l[l == 0] = rng.choice([0.0, -0.0], (l == 0).sum())
    l = l.astype(np.float16 if kind == 16 else np.float32)
    if how == "masked":
        lowest = np.finfo(l.dtype).min
        l[rng.random((M, E)) < 0.4] = -np.inf
        l[rng.random((M, E)) < 0.1] = lowest
        l[::5] = -np.inf
        l[1::7] = lowest
    return l


def weight_tol(l, w):
    """exp to 2^-22 of itself and its argument's rounding, a sum of E of them, two quotients."""
    f = l.astype(np.float64)
    f = np.where(np.isfinite(f) & (f > -1e3), f, np.nan)
    with np.errstate(all="ignore"):
        spread = np.nan_to_num(np.nanmax(np.where(np.isnan(f), -np.inf, f), axis=1) -
                               np.nanmin(np.where(np.isnan(f), np.inf, f), axis=1), posinf=0, neginf=0, nan=0)
    return w * (2.0 ** -20 + (2 * l.shape[1] + 8 * spread[:, None] + 16) * U) + 1e-37


@pytest.mark.parametrize("M,E,T", SIZES)
@pytest.mark.parametrize("kind", [16, 32])
@pytest.mark.parametrize("how", ["plain", "ties", "masked"])
@pytest.mark.parametrize("renorm", [False, True])
def test_route(M, E, T, kind, how, renorm):
    note(f"route M={M} E={E} T={T} bits={kind} {how} renormalise={renorm}")
    rng = np.random.default_rng([96, M, E, T, kind])
    l = logits_of(rng, M, E, kind, how)
    index, weights = w4.w4a16_route(dev(l), T, renormalise=renorm)
    ri, rw, p = oracle.route(l, T, renorm)
    assert np.array_equal(index.cpu().numpy(), ri)
    within("weights", weights, rw, weight_tol(l, rw))
    dw = rng.standard_normal((M, T)).astype(np.float32)
    got = w4.w4a16_route_backward(dev(dw), dev(l), index, weights, renormalise=renorm)
    w = weights.cpu().numpy().astype(np.float64)
    ref = oracle.route_backward(dw, l, ri, w, renorm)
    # sums of T products; p as above; the result's own rounding
    mag = np.abs(dw) * w
    carried = np.zeros((M, E))
    np.add.at(carried, (np.arange(M)[:, None], np.where(ri < 0, 0, ri)), mag + w * mag.sum(1, keepdims=True))
    if not renorm:
        carried += p * mag.sum(1, keepdims=True)
    tol = weight_tol(l, carried) + 2 * (T + 4) * U * carried
    if kind == 16:
        tol = tol + half_tol(np.abs(ref) + tol)
    within("dlogits", got, ref, tol)


def test_route_keeps_nan_and_infinity_to_their_rows():
    note("route with NaN and infinities")
    rng = np.random.default_rng(97)
    l = rng.standard_normal((8, 20)).astype(np.float32)
    clean = l.copy()
    l[1, 3] = np.nan
    l[3, 5] = np.inf
    l[5] = np.nan
    for renorm in (False, True):
        index, weights = w4.w4a16_route(dev(l), 4, renormalise=renorm)
        good_i, good_w = w4.w4a16_route(dev(clean), 4, renormalise=renorm)
        rows = [0, 2, 4, 6, 7]
        assert same(index[rows], good_i[rows]) and same(weights[rows], good_w[rows])
        assert np.isnan(weights.cpu().numpy()[[1, 3]]).all()
        assert index[3, 0].item() == 5 and 3 not in index[1].tolist()
        assert (index[5] == -1).all() and not weights[5].any()


@pytest.mark.parametrize("M,T,N", [(1, 1, 8), (3, 8, 72), (16, 8, 1536), (129, 3, 2056), (5, 17, 4096), (1000, 2, 264)])
def test_combine(M, T, N):
    note(f"combine M={M} T={T} N={N}")
    rng = np.random.default_rng([98, M, T, N])
    y, dout = f16(rng, (M, T, N), 1.5), f16(rng, (M, N), 0.05)
    w = rng.random((M, T)).astype(np.float32)
    w[rng.random((M, T)) < 0.1] = 0
    out = w4.w4a16_experts_combine(dev(y), dev(w))
    ref = oracle.experts_combine(y, w)
    mag = oracle.experts_combine(np.abs(y), w)
    within("out", out, ref, 2 * T * U * mag + half_tol(ref))
    dy, dw = w4.w4a16_experts_combine_backward(dev(dout), dev(y), dev(w))
    rdy, rdw = oracle.experts_combine_backward(dout, y, w)
    within("dy", dy, rdy, U * np.abs(rdy) + half_tol(rdy))
    mag = oracle.experts_combine_backward(np.abs(dout), np.abs(y), w)[1]
    within("dweights", dw, rdw, 2 * N * U * mag + 1e-45)
