"""The float64 oracle of the mixtures of experts and of the vocabulary head's loss: choices
against a plain sort, gradients against central differences."""

import numpy as np
import pytest

import oracle


def difference(f, a, direction, h=1e-5):
    return (f(a + h * direction) - f(a - h * direction)) / (2 * h)


# central differences at h: h^2 / 6 of the third derivative (of order 10 here) and 2^-52 / h of the values
def close(got, ref, size=1.0):
    assert abs(got - ref) <= 1e-7 * (size + abs(ref)), (got, ref)


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("T", [1, 3, 9])
def test_route_and_its_gradient(renorm, T):
    rng = np.random.default_rng(7)
    M, E = 6, 9
    l = rng.standard_normal((M, E))
    l[2, 1] = -np.inf
    index, weights, p = oracle.route(l, T, renorm)
    for m in range(M):
        n = min(T, E - (m == 2))
        assert list(index[m, :n]) == sorted(range(E), key=lambda j: (-l[m, j], j))[:n]
        assert (index[m, n:] == -1).all() and not weights[m, n:].any()
        e = np.exp(l[m] - l[m].max())
        want = (e / e.sum())[index[m, :n]]
        np.testing.assert_allclose(weights[m, :n], want / want.sum() if renorm else want, rtol=1e-13)
        np.testing.assert_allclose(p[m].sum(), 1.0, rtol=1e-13)
    dw = rng.standard_normal((M, T))
    dl = oracle.route_backward(dw, l, index, weights, renorm)
    direction = np.where(np.isfinite(l), rng.standard_normal((M, E)), 0.0)
    step = np.where(np.isfinite(l), direction, 0.0)

    def f(a):
        i, w, _ = oracle.route(a, T, renorm)
        assert np.array_equal(i, index)
        return (dw * w).sum()
    close((dl * step).sum(), difference(f, l, step))


def test_route_breaks_ties_by_index_and_leaves_masked_rows_empty():
    l = np.zeros((3, 5))
    l[1] = -np.inf
    l[2, 0] = np.nan
    index, weights, _ = oracle.route(l, 3)
    assert list(index[0]) == [0, 1, 2] and list(index[1]) == [-1, -1, -1] and list(index[2]) == [1, 2, 3]
    assert np.allclose(weights[0], 1 / 3) and not weights[1].any() and np.isnan(weights[2]).all()


def test_same_expert_twice():
    rng = np.random.default_rng(8)
    w = rng.standard_normal((3, 4, 6))
    x = rng.standard_normal((2, 6))
    index = np.array([[1, 1], [2, -1]])
    y = oracle.experts_gemm(x, w, index)
    assert np.allclose(y[0, 0], w[1] @ x[0]) and np.array_equal(y[0, 0], y[0, 1]) and not y[1, 1].any()
    dy = rng.standard_normal((2, 2, 4))
    dx = oracle.experts_backward(dy, w, index)
    np.testing.assert_allclose(dx[0], (dy[0, 0] + dy[0, 1]) @ w[1], rtol=1e-12)
    np.testing.assert_allclose(dx[1], dy[1, 0] @ w[2], rtol=1e-12)


def test_gradients_of_a_mixture():
    rng = np.random.default_rng(9)
    M, T, E, N, K = 5, 2, 4, 6, 8
    w, x = rng.standard_normal((E, N, K)), rng.standard_normal((M, K))
    index = rng.integers(-1, E, (M, T))
    gate, dout = rng.random((M, T)), rng.standard_normal((M, N))

    def f(a, g):
        return (dout * oracle.experts_combine(oracle.experts_gemm(a, w, index), g)).sum()
    y = oracle.experts_gemm(x, w, index)
    dy, dg = oracle.experts_combine_backward(dout, y, gate)
    dx = oracle.experts_backward(dy, w, index)
    d = rng.standard_normal((M, K))
    close((dx * d).sum(), difference(lambda a: f(a, gate), x, d), 10)
    d = rng.standard_normal((M, T))
    close((dg * d).sum(), difference(lambda g: f(x, g), gate, d), 10)


@pytest.mark.parametrize("vocab", [1, 11, None])
def test_head_loss_and_its_gradient(vocab):
    rng = np.random.default_rng(10)
    M, N, K = 5, 16, 6
    w, x = rng.standard_normal((N, K)), rng.standard_normal((M, K))
    V = N if vocab is None else vocab
    target = rng.integers(0, V, M)
    target[1] = -100
    dloss = rng.standard_normal(M)
    loss, lse, coeff = oracle.head_loss(x, w, target, vocab)
    l = x @ w[:V].T
    keep = np.arange(M) != 1
    np.testing.assert_allclose(lse[keep], np.log(np.exp(l).sum(1))[keep], rtol=1e-12)
    np.testing.assert_allclose(loss[keep], (lse - l[np.arange(M), np.where(keep, target, 0)])[keep], rtol=1e-9, atol=1e-12)
    assert loss[1] == lse[1] == 0 and not coeff[1].any()
    dx = oracle.head_loss_backward(dloss, x, w, target, vocab)
    d = rng.standard_normal((M, K))
    close((dx * d).sum(), difference(lambda a: (dloss * oracle.head_loss(a, w, target, vocab)[0]).sum(), x, d), 10)
