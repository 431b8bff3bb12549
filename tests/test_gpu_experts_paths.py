"""Mixtures of experts and the vocabulary head's loss as they are used: a step of all of them
together, on other streams and in graphs, with padded rows, repeated experts, NaN and
infinities in places that must not matter, sizes past 32 bits, and gradients against
differences."""

import numpy as np
import pytest

import oracle
import w4a16_gemm_amd as w4
from experts_common import U, Layers, backward_tol, dev, f16, gemm_tol, half_tol, make_index, same, within
from gpu_common import device, note
from test_gpu_head import dx_tol, loss_tol
from test_gpu_route import weight_tol

pytestmark = pytest.mark.gpu


def _silu(v):
    import torch
    return (torch.nn.functional.silu(v.float())).half()


def _silu_grad(v, d):
    import torch
    f = v.float()
    s = torch.sigmoid(f)
    return (d.float() * (s * (1 + f * (1 - s)))).half()


class Model:
    """A routed block of `up` and `down` experts and a head, its routing matrix in float32."""

    def __init__(self, E=6, hidden=192, inner=320, vocab=1000, T=2, bits=4, seed=0, act=False):
        self.T, self.vocab = T, vocab
        self.up = Layers(E, inner, hidden, bits, 64, act=act, seed=seed, scale=0.01)
        self.down = Layers(E, hidden, inner, bits, 64, sym=True, seed=seed + 1, scale=0.01)
        self.head = Layers(1, vocab + 8, hidden, bits, 64, act=act, seed=seed + 2, experts=False)
        self.router = dev(np.random.default_rng([99, seed]).standard_normal((E, hidden)).astype(np.float32) / 8)

    def step(self, x, target, dloss, stream=None):
        """Forward and backward: every intermediate result, by name."""
        import torch
        r = {}
        s = dict(stream=stream)
        M = x.shape[0]
        r["logits"] = x.float() @ self.router.T
        r["index"], r["weights"] = w4.w4a16_route(r["logits"], self.T, **s)
        r["y1"] = self.up.fn("experts_gemm")(x, *self.up.args, r["index"], **s)
        r["h"] = _silu(r["y1"])
        flat = r["index"].view(-1)
        r["y2"] = self.down.fn("experts_gemm")(r["h"].view(M * self.T, -1), *self.down.args, flat, **s).view(M, self.T, -1)
        r["out"] = w4.w4a16_experts_combine(r["y2"], r["weights"], **s)
        r["z"] = (x.float() + r["out"].float()).half()
        r["loss"], r["lse"] = self.head.fn("head_loss")(r["z"], *self.head.args, target, vocab=self.vocab, **s)
        r["dz"] = self.head.fn("head_loss_backward")(dloss, r["z"], *self.head.args, target, r["lse"], vocab=self.vocab, **s)
        r["dy2"], r["dw"] = w4.w4a16_experts_combine_backward(r["dz"], r["y2"], r["weights"], **s)
        r["dh"] = self.down.fn("experts_backward")(r["dy2"].view(M * self.T, -1), *self.down.args, flat, r["h"].shape[-1], **s)
        r["dy1"] = _silu_grad(r["y1"], r["dh"].view(M, self.T, -1))
        r["dlogits"] = w4.w4a16_route_backward(r["dw"], r["logits"], r["index"], r["weights"], **s)
        r["dx0"] = (r["dz"].float() + r["dlogits"] @ self.router).half()
        r["dx"] = self.up.fn("experts_backward")(r["dy1"], *self.up.args, r["index"], x.shape[1], dx=r["dx0"], **s)
        return r


def _inputs(M, hidden, vocab, seed):
    rng = np.random.default_rng([100, M, seed])
    target = rng.integers(0, vocab, M).astype(np.int32)
    target[rng.random(M) < 0.2] = -100
    return f16(rng, (M, hidden)), target, rng.uniform(0.5, 8, M).astype(np.float32)


@pytest.mark.parametrize("M,bits,act", [(1, 4, False), (37, 4, False), (400, 4, True), (210, 8, False)])
def test_step(M, bits, act):
    """Every operator's result of a whole step against the oracle at the values that it was given."""
    note(f"step M={M} bits={bits} act={act}")
    m = Model(bits=bits, act=act)
    x, target, dloss = _inputs(M, 192, m.vocab, 1)
    r = m.step(dev(x), dev(target), dev(dloss))
    c = {k: v.cpu().numpy() for k, v in r.items()}
    index = c["index"]
    i, w, _ = oracle.route(c["logits"], m.T)
    assert np.array_equal(index, i)
    within("weights", r["weights"], w, weight_tol(c["logits"], w))
    ref = oracle.experts_gemm(x, m.up.W, index)
    within("y1", r["y1"], ref, gemm_tol(x, m.up.W, index, ref))
    h, flat = c["h"].reshape(M * m.T, -1), index.reshape(-1, 1)
    ref = oracle.experts_gemm(h, m.down.W, flat)
    within("y2", r["y2"].view(M * m.T, 1, -1), ref, gemm_tol(h, m.down.W, flat, ref))
    ref = oracle.experts_combine(c["y2"], c["weights"])
    within("out", r["out"], ref, 2 * m.T * U * oracle.experts_combine(np.abs(c["y2"]), c["weights"]) + half_tol(ref))
    W = m.head.W[0]
    loss, lse, coeff = oracle.head_loss(c["z"], W, target, m.vocab)
    tol = loss_tol(c["z"], W[:m.vocab], lse)
    within("loss", r["loss"], loss, tol[0])
    within("lse", r["lse"], lse, tol[1])
    ref = oracle.head_loss_backward(dloss, c["z"], W, target, m.vocab)
    # dx_tol takes a float32 rounding of the exact lse; this one has the forward's error, in both
    within("dz", r["dz"], ref, 2 * dx_tol(dloss, c["z"], W[:m.vocab], target, lse, coeff, ref))
    dy2, dw = oracle.experts_combine_backward(c["dz"], c["y2"], c["weights"])
    within("dy2", r["dy2"], dy2, U * np.abs(dy2) + half_tol(dy2))
    within("dw", r["dw"], dw, 2 * 192 * U * oracle.experts_combine_backward(np.abs(c["dz"]), np.abs(c["y2"]), c["weights"])[1] + 1e-45)
    d = c["dy2"].reshape(M * m.T, 1, -1)
    ref = oracle.experts_backward(d, m.down.W, flat)
    within("dh", r["dh"], ref, backward_tol(d, m.down.W, flat, None, ref))
    ref = oracle.experts_backward(c["dy1"], m.up.W, index, c["dx0"])
    within("dx", r["dx"], ref, backward_tol(c["dy1"], m.up.W, index, c["dx0"], ref))
    ref = oracle.route_backward(c["dw"], c["logits"], index, c["weights"])
    mag = np.abs(c["dw"]) * c["weights"]
    carried = np.zeros(c["logits"].shape)
    np.add.at(carried, (np.arange(M)[:, None], index), mag + c["weights"] * mag.sum(1, keepdims=True))
    within("dlogits", r["dlogits"], ref, 2 * (m.T + 4) * U * carried + 1e-45)


@pytest.mark.parametrize("M", [3, 300])
def test_two_graphs_of_a_step(M):
    """Two captured steps with workspaces of their own, replayed at once on two streams, with
    eager steps and other inputs between the replays."""
    import torch
    note(f"graphs of a step M={M}")
    models = [Model(seed=0), Model(seed=5, bits=8)]
    held, graphs, outs = [], [], []
    for m in models:
        t = [dev(a) for a in _inputs(M, 192, m.vocab, 2)]
        m.step(*t)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(m.step(*t))
        held.append(t)
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for replay in range(4):
        for m, t in zip(models, held):
            for a, b in zip(t, _inputs(M, 192, m.vocab, 10 + replay)):
                a.copy_(dev(b))
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for m, t, o in zip(models, held, outs):
            want = m.step(*t)
            torch.cuda.synchronize()
            for k, v in want.items():
                assert same(o[k], v), (replay, k)


def test_two_streams_at_once():
    import torch
    note("two streams")
    models = [Model(seed=0), Model(seed=5, bits=8)]
    held = [[dev(a) for a in _inputs(260, 192, m.vocab, 3 + i)] for i, m in enumerate(models)]
    want = [m.step(*t) for m, t in zip(models, held)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(4):
        got = []
        for m, t, s in zip(models, held, streams):
            with torch.cuda.stream(s):
                got.append(m.step(*t))
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert all(same(g[k], w[k]) for k in w)


def test_stream_argument():
    """A call on a stream of its own, of tensors made on the current one."""
    import torch
    note("stream argument")
    rng = np.random.default_rng(101)
    layers = Layers(4, 264, 128)
    x, index = dev(f16(rng, (50, 128))), dev(make_index(rng, 50, 2, 4, "mixed"))
    want = w4.w4a16_experts_gemm(x, *layers.args, index)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = torch.empty_like(want)
    got = w4.w4a16_experts_gemm(x, *layers.args, index, out=out, stream=s)
    s.synchronize()
    assert got.data_ptr() == out.data_ptr() and same(out, want)


# few rows; tiles of 64; of 256 and a remainder
ROWS = [(20, 2, 8), (150, 2, 4), (900, 2, 3)]


@pytest.mark.parametrize("M,T,E", ROWS)
@pytest.mark.parametrize("bits", [4, 8])
def test_nan_and_infinity_stay_in_their_rows(M, T, E, bits):
    import torch
    note(f"NaN rows M={M} bits={bits}")
    rng = np.random.default_rng([102, M, bits])
    layers = Layers(E, 528, 192, bits, 64)
    index = make_index(rng, M, T, E, "mixed")
    x, dy = f16(rng, (M, 192)), f16(rng, (M, T, 528), 0.05)
    y = layers.fn("experts_gemm")(dev(x), *layers.args, dev(index))
    dx = layers.fn("experts_backward")(dev(dy), *layers.args, dev(index), 192)
    bad = rng.choice(M, M // 5, replace=False)
    x[bad[::2], 7], x[bad[1::2], 9] = np.nan, np.inf
    dy[bad] = np.nan
    dy[index < 0] = np.nan          # slots without an expert: not read
    keep = dev(~np.isin(np.arange(M), bad))
    y2 = layers.fn("experts_gemm")(dev(x), *layers.args, dev(index))
    dx2 = layers.fn("experts_backward")(dev(dy), *layers.args, dev(index), 192)
    assert same(y2[keep], y[keep]) and same(dx2[keep], dx[keep])
    used = dev(index >= 0)
    assert not y2[~used].any()
    assert not torch.isfinite(y2[~keep][used[~keep]]).any()
    assert torch.isnan(dx2[~keep][used[~keep].any(1)]).all()


@pytest.mark.parametrize("M,T,E", ROWS)
def test_experts_that_are_not_chosen_do_not_matter(M, T, E):
    """Layers of NaN scales, chosen by nobody; the same expert in every slot of a row."""
    note(f"unused experts M={M}")
    rng = np.random.default_rng([103, M])
    layers = Layers(E, 264, 128)
    index = np.repeat(rng.integers(0, E - 1, (M, 1)), T, 1).astype(np.int32)
    q, s, z, _, group = layers.args
    s = s.clone()
    s[E - 1] = float("nan")
    x, dy = f16(rng, (M, 128)), f16(rng, (M, T, 264), 0.05)
    y = w4.w4a16_experts_gemm(dev(x), q, s, z, None, group, dev(index))
    ref = oracle.experts_gemm(x, layers.W, index)
    within("y", y, ref, gemm_tol(x, layers.W, index, ref))
    assert all(same(y[:, t], y[:, 0]) for t in range(T))
    dx = w4.w4a16_experts_backward(dev(dy), q, s, z, None, group, dev(index), 128)
    ref = oracle.experts_backward(dy, layers.W, index)
    within("dx", dx, ref, backward_tol(dy, layers.W, index, None, ref))


@pytest.mark.parametrize("M", [5, 300])
@pytest.mark.parametrize("vocab", [257, 511, 760])
@pytest.mark.parametrize("bits", [4, 8])
def test_padding_of_the_vocabulary_takes_no_part(M, vocab, bits):
    """Rows of weights past the vocabulary that are infinite or NaN."""
    note(f"vocabulary padding M={M} vocab={vocab} bits={bits}")
    rng = np.random.default_rng([104, M, vocab])
    layer = Layers(1, 768, 128, bits, 64, experts=False)
    q, s, z, g, group = layer.args
    wild = s.clone()
    wild[:, vocab:] = float("inf")
    wild[:, vocab + 1::2] = float("nan")
    x, target = dev(f16(rng, (M, 128), 2.0)), dev(rng.integers(0, vocab, M).astype(np.int32))
    dloss = dev(np.ones(M, np.float32))
    loss, lse = layer.fn("head_loss")(x, q, s, z, g, group, target, vocab=vocab)
    loss2, lse2 = layer.fn("head_loss")(x, q, wild, z, g, group, target, vocab=vocab)
    assert same(loss, loss2) and same(lse, lse2)
    dx = layer.fn("head_loss_backward")(dloss, x, q, s, z, g, group, target, lse, vocab=vocab)
    dx2 = layer.fn("head_loss_backward")(dloss, x, q, wild, z, g, group, target, lse, vocab=vocab)
    assert same(dx, dx2)


@pytest.mark.parametrize("M", [40, 300])
def test_wild_rows_of_the_loss_stay_alone(M):
    import torch
    note(f"loss with NaN rows M={M}")
    rng = np.random.default_rng([105, M])
    layer = Layers(1, 1032, 128, 4, 64, experts=False)
    x, target = f16(rng, (M, 128), 2.0), rng.integers(0, 1032, M).astype(np.int32)
    run = lambda a: layer.fn("head_loss")(dev(a), *layer.args, dev(target))   # noqa: E731
    back = lambda a, lse: layer.fn("head_loss_backward")(dev(np.ones(M, np.float32)), dev(a), *layer.args,   # noqa: E731
                                                         dev(target), lse)
    loss, lse = run(x)
    dx = back(x, lse)
    bad = x.copy()
    bad[3, 5], bad[11, 0], bad[17] = np.nan, np.inf, -np.inf
    wild = [3, 11, 17]
    keep = [m for m in range(M) if m not in wild]
    loss2, lse2 = run(bad)
    dx2 = back(bad, lse2)
    assert same(loss2[keep], loss[keep]) and same(lse2[keep], lse[keep]) and same(dx2[keep], dx[keep])
    assert not torch.isfinite(loss2[wild]).any() and not torch.isfinite(dx2[wild]).any()


def test_loss_of_more_rows_than_one_pass_takes():
    note("loss of 33000 rows")
    rng = np.random.default_rng(106)
    M, N, K = 33000, 264, 64
    layer = Layers(1, N, K, 4, 64, act=True, experts=False)
    x, target = f16(rng, (M, K), 2.0), rng.integers(-1, N, M).astype(np.int32)
    loss, lse = layer.fn("head_loss")(dev(x), *layer.args, dev(target))
    dloss = np.full(M, 4.0, np.float32)
    dx = layer.fn("head_loss_backward")(dev(dloss), dev(x), *layer.args, dev(target), lse)
    rows = np.r_[0:40, 32700:32840, 32960:33000]
    W = layer.W[0]
    rl, rs, coeff = oracle.head_loss(x[rows], W, target[rows])
    tol = loss_tol(x[rows], W, rs)
    within("loss", loss[dev(rows)], rl, tol[0])
    within("lse", lse[dev(rows)], rs, tol[1])
    ref = oracle.head_loss_backward(dloss[rows], x[rows], W, target[rows])
    within("dx", dx[dev(rows)], ref, 2 * dx_tol(dloss[rows], x[rows], W, target[rows], rs, coeff, ref))


def test_outputs_past_32_bits():
    """More than 2^31 outputs: products, and their weighted sum."""
    import torch
    note("experts of 2.3e9 outputs")
    rng = np.random.default_rng(107)
    M, T, E, N, K = 140000, 2, 3, 8192, 64
    layers = Layers(E, N, K, 4, 64)
    x, index = f16(rng, (M, K)), make_index(rng, M, T, E, "distinct")
    y = w4.w4a16_experts_gemm(dev(x), *layers.args, dev(index))
    rows = np.r_[0:3, 70000:70003, M - 3:M]
    ref = oracle.experts_gemm(x[rows], layers.W, index[rows])
    within("y", y[dev(rows)], ref, gemm_tol(x[rows], layers.W, index[rows], ref))
    w = rng.random((M, T)).astype(np.float32)
    out = w4.w4a16_experts_combine(y, dev(w))
    part = y[dev(rows)].cpu().numpy()
    ref = oracle.experts_combine(part, w[rows])
    within("out", out[dev(rows)], ref, 2 * T * U * oracle.experts_combine(np.abs(part), w[rows]) + half_tol(ref))
    del out
    dout = torch.ones((M, N), dtype=torch.float16, device=device())
    dy, dw = w4.w4a16_experts_combine_backward(dout, y, dev(w))
    rdy, rdw = oracle.experts_combine_backward(np.ones((len(rows), N)), part, w[rows])
    within("dy", dy[dev(rows)], rdy, half_tol(rdy))
    within("dw", dw[dev(rows)], rdw, 2 * N * U * oracle.experts_combine_backward(np.ones((len(rows), N)), np.abs(part), w[rows])[1])


# --- gradients against differences ------------------------------------------------------------


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("M,T,E", ROWS)
def test_gradient_of_products_against_differences(M, T, E, bits):
    """Small integers: with at most 9 units in a row of x, 10 in one of dy, and weights within
    191, products and gradients stay below 2048 and are exact, and so is
    <dy, y(x + d) - y(x)> = <dx, d>."""
    note(f"differences of products M={M} bits={bits}")
    rng = np.random.default_rng([108, M, bits])
    N, K = 48, 64
    layers = Layers(E, N, K, bits, 64)
    q, s, z, g, group = layers.args
    s = s * 0 + 1

    def units(rows, cols, n):
        a = np.zeros((rows, cols), np.float16)
        a[np.arange(rows)[:, None], np.argsort(rng.random((rows, cols)), axis=1)[:, :n]] = rng.choice([-1, 1], (rows, n))
        return a
    index = dev(make_index(rng, M, T, E, "mixed"))
    x, d, dy = units(M, K, 7), units(M, K, 2), units(M * T, N, 5).reshape(M, T, N)
    run = lambda a: layers.fn("experts_gemm")(dev(a), q, s, z, g, group, index).double()   # noqa: E731
    moved = run(x + d) - run(x)
    dx = layers.fn("experts_backward")(dev(dy), q, s, z, g, group, index, K).double()
    assert (dev(dy).double() * moved).sum().item() == (dx * dev(d).double()).sum().item()
    assert dx.any()


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("E,T", [(8, 2), (64, 8), (300, 20)])
def test_gradient_of_routing_against_differences(E, T, renorm):
    """Steps of h = 2^-8 along d, |d| <= 1: the third derivative of a softmax weight is at most
    18 there, so a central difference is off by 3 h^2; its two weights by the bound of the
    weights each."""
    note(f"differences of routing E={E} T={T}")
    rng = np.random.default_rng([109, E])
    M, h = 50, 2.0 ** -8
    # logits apart by 2^-4 and more: no step changes the choice
    l = (np.argsort(rng.random((M, E)), axis=1) * 2.0 ** -4).astype(np.float32)
    d = rng.uniform(-1, 1, (M, E)).astype(np.float32)
    dw = rng.standard_normal((M, T)).astype(np.float32)
    up, down, at = ((l + s * h * d).astype(np.float32) for s in (1, -1, 0))
    index, weights = w4.w4a16_route(dev(at), T, renormalise=renorm)
    runs = [w4.w4a16_route(dev(a), T, renormalise=renorm) for a in (up, down)]
    assert all(same(r[0], index) for r in runs)
    step = (up.astype(np.float64) - down) / 2
    got = w4.w4a16_route_backward(dev(dw), dev(at), index, weights, renormalise=renorm).cpu().numpy().astype(np.float64)
    moved = (runs[0][1].double() - runs[1][1].double()).cpu().numpy() / 2
    w = weights.cpu().numpy().astype(np.float64)
    tol = np.abs(dw) * (weight_tol(up, w * 1.01) + 3 * h ** 3 + 1e-6 * h)
    assert (np.abs((got * step).sum(1) - (dw * moved).sum(1)) <= tol.sum(1)).all()


@pytest.mark.parametrize("bits,act", [(4, False), (4, True), (8, False)])
def test_gradient_of_the_loss_against_differences(bits, act):
    """Steps of h = 2^-3 along d of -1, 0 and 1.  The third cumulant of logits' slopes within a
    range L is at most L^3 / (6 sqrt 3), so a central difference is off by h^2 L^3 / (36 sqrt 3);
    its losses by their own bound, the gradient by its."""
    note(f"differences of the loss bits={bits} act={act}")
    rng = np.random.default_rng([110, bits])
    M, N, K, h = 60, 2064, 192, 2.0 ** -3
    layer = Layers(1, N, K, bits, 64, act=act, experts=False, scale=0.02)
    W = layer.W[0].astype(np.float64)
    x = (rng.integers(-8, 9, (M, K)) / 8).astype(np.float16)
    d = (rng.integers(-1, 2, (M, K)) * (rng.random((M, K)) < 0.05)).astype(np.float16)
    target = rng.integers(0, N, M).astype(np.int32)
    run = lambda a: layer.fn("head_loss")(dev(a), *layer.args, dev(target))   # noqa: E731
    _, lse = run(x)
    dloss = np.ones(M, np.float32)
    dx = layer.fn("head_loss_backward")(dev(dloss), dev(x), *layer.args, dev(target), lse).cpu().numpy().astype(np.float64)
    up, down = (run((x + s * np.float16(h) * d).astype(np.float16))[0].cpu().numpy().astype(np.float64) for s in (1, -1))
    slope = W @ d.astype(np.float64).T
    L = slope.max(axis=0) - slope.min(axis=0)
    rl, rs, coeff = oracle.head_loss(x, W, target)
    ref = oracle.head_loss_backward(dloss, x, W, target)
    tol = (h ** 2 * L ** 3 / (36 * 3 ** 0.5) + 1.1 * loss_tol(np.abs(x) + h, W, rs + 1)[0] / h
           + (2 * dx_tol(dloss, x, W, target, rs, coeff, ref) * np.abs(d)).sum(1))
    err = np.abs((dx * d).sum(1) - (up - down) / (2 * h))
    assert (err <= tol).all(), (err / tol).max()
    assert np.median(np.abs((dx * d).sum(1))) > 3 * np.median(tol)     # the comparison says something


# --- refusals on the device -------------------------------------------------------------------


def test_refusals_on_the_device():
    import torch
    note("refusals")
    dv = device()
    f, i32 = torch.float16, torch.int32
    E, M, T, N, K = 3, 6, 2, 64, 128
    layers = Layers(E, N, K)
    x, y = torch.zeros((M, K), dtype=f, device=dv), torch.zeros((M, T, N), dtype=f, device=dv)
    index, weights = torch.zeros((M, T), dtype=i32, device=dv), torch.zeros((M, T), device=dv)
    logits = torch.zeros((M, 8), device=dv)
    head = Layers(1, N, K, experts=False)
    target, rows = torch.zeros(M, dtype=i32, device=dv), torch.zeros(M, device=dv)
    a = layers.args
    buf = torch.zeros(4 * M * T * N, dtype=f, device=dv)
    part = buf[:M * T * N].view(M, T, N)
    for bad in [
        lambda: w4.w4a16_experts_gemm(x, *a, index, out=torch.empty((M, T, N + 8), dtype=f, device=dv)),
        lambda: w4.w4a16_experts_gemm(x, *a, index.cpu()),
        lambda: w4.w4a16_experts_gemm(x[:, ::2], *a, index),
        lambda: w4.w4a16_experts_gemm(x.float(), *a, index),
        lambda: w4.w4a16_experts_gemm(x, *a, index.long()),
        lambda: w4.w4a16_experts_gemm(x, *a, index[:-1]),
        lambda: w4.w4a16_experts_gemm(x[:0], *a, index[:0]),
        lambda: w4.w8a16_experts_gemm(x, *a, index),
        lambda: w4.w4a16_experts_gemm(buf[:M * K].view(M, K), *a, index, out=part),
        lambda: w4.w4a16_experts_backward(part, *a, index, K, out=buf[8:8 + M * K].view(M, K)),
        lambda: w4.w4a16_experts_backward(y, *a, index, K + 1),
        lambda: w4.w4a16_experts_backward(y, *a, None, K),
        lambda: w4.w4a16_experts_backward(y, *a, index, K, dx=x[1:]),
        lambda: w4.w4a16_experts_combine(part, weights, out=buf[16:16 + M * N].view(M, N)),
        lambda: w4.w4a16_experts_combine(y, weights.double()),
        lambda: w4.w4a16_route(logits, 9),
        lambda: w4.w4a16_route(logits, 0),
        lambda: w4.w4a16_route(logits.bfloat16(), 2),
        lambda: w4.w4a16_route(logits[:, ::2], 2),
        lambda: w4.w4a16_route(logits, 8, weights=logits),
        lambda: w4.w4a16_route_backward(weights, logits, index, weights, out=logits),
        lambda: w4.w4a16_head_loss(x, *head.args, target, vocab=0),
        lambda: w4.w4a16_head_loss(x, *head.args, target, vocab=N + 1),
        lambda: w4.w4a16_head_loss(x, *head.args, target, loss=rows, lse=rows),
        lambda: w4.w4a16_head_loss_backward(rows, x, *head.args, target, rows, out=x),
        lambda: w4.w4a16_gemm_backward(y[:, 0], *head.args, K),
    ]:
        with pytest.raises((ValueError, TypeError, w4.W4A16Error)):
            bad()


@pytest.mark.parametrize("M", [1, 300])
def test_gradient_of_the_layer_is_that_of_its_restored_weights(M):
    """Against dy times the layer's own w4a16_dequant, and in place on a gradient that is there."""
    note(f"layer gradient M={M}")
    rng = np.random.default_rng([111, M])
    N, K = 520, 448
    layer = Layers(1, N, K, 4, 64, act=True, experts=False)
    dy, dx0 = f16(rng, (M, N), 0.05), f16(rng, (M, K), 0.05)
    out = dev(dx0)
    got = w4.w4a16_gemm_backward(dev(dy), *layer.args, K, dx=out, out=out)
    W = w4.w4a16_dequant(*layer.args, K).cpu().numpy()
    index = np.zeros((M, 1), np.int32)
    ref = oracle.experts_backward(dy[:, None], W[None], index, dx0)
    within("dx", got, ref, backward_tol(dy[:, None], W[None], index, dx0, ref))


@pytest.mark.parametrize("M,N,vocab,K,act,none", [(37, 140008, 140001, 64, False, 0.3), (64, 151936, 151936, 128, False, 0.0),
                                                  (1, 135000, 134999, 192, False, 0.0), (5, 140008, 140008, 64, False, 1.0),
                                                  (100, 70000, 69990, 64, False, 0.1), (50, 140008, 140008, 64, True, 0.2)])
def test_loss_of_few_rows_against_wide_heads(M, N, vocab, K, act, none):
    note(f"few rows, wide head M={M} N={N} K={K} act={act}")
    rng = np.random.default_rng([112, M, N])
    layer = Layers(1, N, K, 4, 64, act=act, experts=False)
    x, target = f16(rng, (M, K), 2.0), rng.integers(0, vocab, M).astype(np.int32)
    target[rng.random(M) < none] = -100
    got = w4.w4a16_head_loss(dev(x), *layer.args, dev(target), vocab=vocab)
    loss, lse, _ = oracle.head_loss(x, layer.W[0], target, vocab)
    tol = loss_tol(x, layer.W[0][:vocab], lse)
    within("loss", got[0], loss, tol[0])
    within("lse", got[1], lse, tol[1])
    again = w4.w4a16_head_loss(dev(x), *layer.args, dev(target), vocab=vocab)
    assert same(got[0], again[0]) and same(got[1], again[1])


# --- every kind of tile: full and small ones, alone and two to a compute unit -------------------

LARGE = [
    # M, T, E, N, K, bits, group, sym, act, index
    (1138, 1, 20, 4672, 128, 4, 64, False, False, "distinct"),
    (1138, 1, 20, 4672, 128, 8, 64, False, False, "mixed"),
    (500, 2, 3, 16400, 64, 4, 32, False, False, "skewed"),
    (500, 2, 3, 16400, 64, 8, 64, True, False, "distinct"),
    (937, 1, 12, 2896, 192, 4, 64, False, True, "padded"),
    (937, 1, 12, 2896, 192, 8, 64, False, False, "distinct"),
    (2010, 2, 40, 528, 128, 4, 128, False, False, "mixed"),
    (2010, 2, 40, 528, 128, 8, 128, False, False, "padded"),
    (300, 1, 1, 5008, 320, 8, 64, False, False, "one"),
    # few rows: long walks, many slots
    (100, 2, 16, 520, 4096, 4, 128, False, False, "distinct"),
    (100, 2, 16, 528, 4224, 8, 64, False, False, "mixed"),
    (9, 3, 8, 528, 4096, 8, 128, False, True, "distinct"),
]
BACK = [
    (66, 1, 40, 528, 2048, 4, 64, False, False, "distinct"),
    (66, 1, 40, 528, 2048, 8, 64, False, False, "mixed"),
    (502, 2, 20, 528, 4096, 4, 64, False, False, "mixed"),
    (502, 2, 20, 528, 4096, 8, 64, True, False, "padded"),
    (1004, 1, 8, 272, 4096, 4, 128, False, True, "distinct"),
    (1000, 2, 8, 272, 4096, 8, 128, False, False, "skewed"),
    (1600, 1, 8, 144, 4096, 4, 128, False, False, "distinct"),
    (2000, 2, 3, 144, 4096, 8, 128, False, True, "distinct"),
    (3000, 1, 2, 1552, 448, 4, 64, False, False, "distinct"),
    (700, 1, 2, 4112, 448, 8, 64, False, False, "skewed"),
]


def _some(rng, M, n=150):
    return np.sort(rng.choice(M, min(M, n), replace=False))


@pytest.mark.parametrize("shape", LARGE, ids=str)
def test_products_in_every_tile(shape):
    M, T, E, N, K, bits, group, sym, act, how = shape
    note(f"tiles {shape}")
    rng = np.random.default_rng([113, M, N, K, bits])
    layers = Layers(E, N, K, bits, group, sym, act)
    x, index = f16(rng, (M, K)), make_index(rng, M, T, E, how)
    y = layers.fn("experts_gemm")(dev(x), *layers.args, dev(index))
    rows = _some(rng, M)
    ref = oracle.experts_gemm(x[rows], layers.W, index[rows])
    within("y", y[dev(rows)], ref, gemm_tol(x[rows], layers.W, index[rows], ref))
    assert not y[dev(index < 0)].any()
    # the same rows in other tiles
    order = rng.permutation(M)
    again = layers.fn("experts_gemm")(dev(x[order]), *layers.args, dev(index[order]))
    within("again", again[dev(np.argsort(order)[rows])], ref, gemm_tol(x[rows], layers.W, index[rows], ref))


@pytest.mark.parametrize("shape", BACK, ids=str)
@pytest.mark.parametrize("add", [False, True], ids=["alone", "added"])
def test_products_back_in_every_tile(shape, add):
    M, T, E, N, K, bits, group, sym, act, how = shape
    note(f"tiles back {shape} added={add}")
    rng = np.random.default_rng([114, M, N, K, bits])
    layers = Layers(E, N, K, bits, group, sym, act)
    dy, index = f16(rng, (M, T, N), 0.05), make_index(rng, M, T, E, how)
    dx0 = f16(rng, (M, K), 0.05) if add else None
    run = lambda: layers.fn("experts_backward")(dev(dy), *layers.args, dev(index), K, dx=dev(dx0))   # noqa: E731
    dx = run()
    rows = _some(rng, M)
    part = dx0[rows] if add else None
    ref = oracle.experts_backward(dy[rows], layers.W, index[rows], part)
    within("dx", dx[dev(rows)], ref, backward_tol(dy[rows], layers.W, index[rows], part, ref))
    assert same(dx, run())


@pytest.mark.parametrize("M,N,vocab,K,act", [(803, 16512, 16500, 64, False), (401, 18896, 18890, 128, False),
                                             (5493, 528, 520, 64, False), (1200, 8208, 8208, 128, True),
                                             (3000, 2064, 2050, 64, False)])
@pytest.mark.parametrize("bits", [4, 8])
def test_loss_in_every_tile(M, N, vocab, K, act, bits):
    note(f"loss tiles M={M} N={N} K={K} bits={bits}")
    rng = np.random.default_rng([115, M, N, bits])
    layer = Layers(1, N, K, bits, 64, act=act, experts=False)
    x, target = f16(rng, (M, K), 2.0), rng.integers(0, vocab, M).astype(np.int32)
    target[rng.random(M) < 0.2] = -100
    dloss = rng.uniform(0.1, 8, M).astype(np.float32)
    loss, lse = layer.fn("head_loss")(dev(x), *layer.args, dev(target), vocab=vocab)
    dx = layer.fn("head_loss_backward")(dev(dloss), dev(x), *layer.args, dev(target), lse, vocab=vocab)
    rows, W = _some(rng, M, 120), layer.W[0]
    rl, rs, coeff = oracle.head_loss(x[rows], W, target[rows], vocab)
    tol = loss_tol(x[rows], W[:vocab], rs)
    within("loss", loss[dev(rows)], rl, tol[0])
    within("lse", lse[dev(rows)], rs, tol[1])
    ref = oracle.head_loss_backward(dloss[rows], x[rows], W, target[rows], vocab)
    within("dx", dx[dev(rows)], ref, 2 * dx_tol(dloss[rows], x[rows], W[:vocab], target[rows], rs, coeff, ref))
    assert same(dx, layer.fn("head_loss_backward")(dev(dloss), dev(x), *layer.args, dev(target), lse, vocab=vocab))


@pytest.mark.parametrize("E", [3, 200])
def test_many_slots(E):
    """More than 2^20 slots, rows and their routing."""
    note(f"many slots E={E}")
    rng = np.random.default_rng([116, E])
    M, T, N, K = 400000, 3, 64, 64
    layers = Layers(E, N, K, 4, 64, sym=True)
    logits = rng.standard_normal((M, E), dtype=np.float32)
    index, weights = w4.w4a16_route(dev(logits), T)
    rows = np.r_[0:20, M // 2:M // 2 + 20, M - 20:M]
    ri, rw, _ = oracle.route(logits[rows], T)
    assert np.array_equal(index[dev(rows)].cpu().numpy(), ri)
    within("weights", weights[dev(rows)], rw, weight_tol(logits[rows], rw))
    x = f16(rng, (M, K))
    y = w4.w4a16_experts_gemm(dev(x), *layers.args, index)
    ref = oracle.experts_gemm(x[rows], layers.W, ri)
    within("y", y[dev(rows)], ref, gemm_tol(x[rows], layers.W, ri, ref))
    dx = w4.w4a16_experts_backward(y, *layers.args, index, K)
    dy = y[dev(rows)].cpu().numpy()
    ref = oracle.experts_backward(dy, layers.W, ri)
    within("dx", dx[dev(rows)], ref, backward_tol(dy, layers.W, ri, None, ref))


@pytest.mark.parametrize("E,how", [(5, "mixed"), (512, "padded"), (1, "one"), (7, "skewed"), (4, "none")])
def test_ragged_groups_of_many_slots(E, how):
    """Slots that several workgroups sort."""
    note(f"many ragged slots E={E} {how}")
    rng = np.random.default_rng([117, E])
    M, T, N, K = (30011, 1 if E == 1 else 3, 64, 64)
    layers = Layers(E, N, K, 4, 64)
    index = make_index(rng, M, T, E, how)
    x, dx0 = f16(rng, (M, K)), f16(rng, (M, K), 0.05)
    y = w4.w4a16_experts_gemm(dev(x), *layers.args, dev(index))
    ref = oracle.experts_gemm(x, layers.W, index)
    within("y", y, ref, gemm_tol(x, layers.W, index, ref))
    dy = f16(rng, (M, T, N), 0.05)
    dx = w4.w4a16_experts_backward(dev(dy), *layers.args, dev(index), K, dx=dev(dx0))
    ref = oracle.experts_backward(dy, layers.W, index, dx0)
    within("dx", dx, ref, backward_tol(dy, layers.W, index, dx0, ref))
