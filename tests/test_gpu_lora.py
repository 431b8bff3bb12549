"""Low-rank adapters on the GPU against the float64 oracle: forward and gradients over odd
sizes, rank and row orders, rows and adapters that hold nothing, values beyond binary16,
NaN and infinities that must not spread, other streams, graphs, and the run of a training
step around the quantised layer.

Tolerances are bounds, not fits.  u = 2^-24.  An fp32 sum of n products in any order is
within 2 n u of sum |p| (the factor 2 covers matrix instructions that add several products
with truncation); an intermediate enters the second product with 2^-22 of itself plus
2^-37 of the largest in its row or chunk (two binary16 terms below 2^14); a binary16
result adds 2^-11 of itself and half a subnormal step, 2^-25."""

import numpy as np
import pytest

import oracle
import w4a16_gemm_amd as w4
import workloads as wl
from gpu_common import device, note, product_layer

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def make(M, N, K, R, L, order, bare=0.0, seed=0, x_std=1.0, a_std=None, b_std=0.05, dy_std=0.05):
    rng = np.random.default_rng([91, M, N, K, R, L, seed])
    f16 = lambda shape, std: (rng.standard_normal(shape) * std).astype(np.float16)   # noqa: E731
    d = {"y": f16((M, N), 1.5), "x": f16((M, K), x_std), "a": f16((L, R, K), K ** -0.5 if a_std is None else a_std),
         "b": f16((L, N, R), b_std), "dy": f16((M, N), dy_std), "dx0": f16((M, K), 0.05),
         "scaling": rng.uniform(0.25, 2.0, L).astype(np.float32), "index": None}
    if order != "one":
        index = rng.integers(0, L, M)
        if order == "runs":
            index = np.sort(index)
        if order == "last":
            index[:] = L - 1
        index[rng.random(M) < bare] = -1
        if order == "none":
            index[:] = rng.choice([-1, L, -2 ** 31, 2 ** 31 - 1], M)
        d["index"] = index.astype(np.int32)
    return d


def dev(a):
    import torch
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(device())


def bits(t):
    import torch
    return t.contiguous().view({2: torch.int16, 4: torch.int32}[t.element_size()])


def same(a, b):
    import torch
    return torch.equal(bits(a), bits(b))


def magnitudes(d):
    """|.| of every operand, as the inputs of the same formulas."""
    return {k: (np.abs(v.astype(np.float64)) if k not in ("index", "scaling") and v is not None else v) for k, v in d.items()}


def half_tol(ref):
    return 2.0 ** -11 * np.abs(ref) + 2.0 ** -25


def forward_tol(d, ref_out):
    """Tolerances of (out, h)."""
    m = magnitudes(d)
    K, R = d["x"].shape[1], d["a"].shape[1]
    zero = np.zeros_like(m["y"])
    _, h_mag = oracle.lora_forward(zero, m["x"], m["a"], m["b"], d["index"], d["scaling"])
    h_tol = 2 * K * U * h_mag
    _, h = oracle.lora_forward(d["y"], d["x"], d["a"], d["b"], d["index"], d["scaling"])
    h_abs = np.abs(h) + h_tol
    carried = h_tol + (2.0 ** -22 + 2 * (2 * R + 8) * U) * h_abs + 2.0 ** -37 * h_abs.max(axis=1, keepdims=True)
    spread = np.zeros_like(m["y"])
    L = d["a"].shape[0]
    owner = np.zeros(len(h), int) if d["index"] is None else d["index"]
    s = np.ones(L) if d["scaling"] is None else d["scaling"]
    for i in range(L):
        rows = owner == i
        spread[rows] = s[i] * (carried[rows] @ m["b"][i].T)
    return spread + half_tol(np.abs(ref_out) + spread) + 2 * U * np.abs(ref_out), h_tol + 1e-45


def backward_tol(d, h, ref):
    """Tolerances of (dx, da, db)."""
    m = magnitudes(d)
    h_mag = np.abs(h)
    M, N = d["dy"].shape
    R, L = d["a"].shape[1], d["a"].shape[0]
    owner = np.zeros(M, int) if d["index"] is None else d["index"]
    s = np.ones(L) if d["scaling"] is None else np.asarray(d["scaling"], np.float64)
    dx = np.zeros(m["x"].shape)
    da, db = np.zeros(m["a"].shape), np.zeros(m["b"].shape)
    for i in range(L):
        rows = np.nonzero(owner == i)[0]
        if rows.size == 0:
            continue
        g_mag = m["dy"][rows] @ m["b"][i]
        g_tol = 2 * N * U * g_mag
        split = lambda v: (2.0 ** -22 + 2 * (2 * max(R, rows.size) + 40) * U) * v   # noqa: E731
        carried = g_tol + split(g_mag) + 2.0 ** -37 * g_mag.max(axis=1, keepdims=True)
        dx[rows] = s[i] * (carried @ m["a"][i])
        # one power of two for the rows of a wavefront: its floor is relative to the largest
        carried = g_tol + split(g_mag) + 2.0 ** -37 * g_mag.max()
        da[i] = s[i] * (carried.T @ m["x"][rows])
        carried = split(h_mag[rows]) + 2.0 ** -37 * h_mag[rows].max()
        db[i] = s[i] * (m["dy"][rows].T @ carried)
    tiny = 1e-45
    return dx + half_tol(np.abs(ref[0]) + dx) + 2 * U * np.abs(ref[0]), da + tiny, db + tiny


def within(name, got, ref, tol):
    got = got.detach().cpu().numpy().astype(np.float64)
    err = np.abs(got - ref)
    bad = ~(err <= tol)
    assert not bad.any(), (f"{name}: {int(bad.sum())} of {bad.size} beyond the bound, worst at "
                           f"{np.unravel_index(np.argmax(np.where(bad, err / tol, 0)), bad.shape)}: "
                           f"{np.nanmax(err / tol):.3g} times")


def forward(d, **kw):
    return w4.w4a16_lora_forward(dev(d["y"]), dev(d["x"]), dev(d["a"]), dev(d["b"]), dev(d["index"]), dev(d["scaling"]), **kw)


def backward(d, h, dx0=True, **kw):
    return w4.w4a16_lora_backward(dev(d["dy"]), dev(d["x"]), dev(d["a"]), dev(d["b"]), h, dev(d["index"]),
                                  dev(d["scaling"]), dx=dev(d["dx0"]) if dx0 else None, **kw)


CASES = [
    # M, N, K, R, L, order, bare: one row; every tile edge around 16, 32 and 64 rows; the
    # last row count the workgroups group themselves (256) and the first beyond it; more
    # adapters than lanes, more rows than the grouping reads at once (8192); channel counts
    # below one step, off every tile, and over several workgroups and slices; ranks at and
    # between the fragment sizes, each with few and with many rows; few channels under many
    # rows (gradients in parts); adapters without rows, rows without an adapter, no index
    # with several adapters; many adapters of few rows each under many channels; numbers of
    # adapters at and beyond those that one, two and three looks of 64 find
    (1, 8, 8, 8, 1, "one", 0), (1, 1536, 1536, 16, 4, "mixed", 0), (2, 136, 40, 8, 3, "mixed", 0),
    (15, 520, 512, 16, 1, "one", 0), (16, 512, 1024, 24, 2, "mixed", 0.2), (17, 1000, 1032, 32, 17, "mixed", 0.1),
    (33, 264, 2048, 40, 5, "runs", 0.2), (63, 640, 264, 48, 100, "mixed", 0.1), (64, 1544, 520, 64, 3, "runs", 0),
    (65, 1544, 520, 64, 3, "runs", 0), (65, 72, 4104, 72, 65, "mixed", 0.5), (127, 2056, 136, 16, 2, "last", 0),
    (200, 520, 776, 128, 6, "mixed", 0.1), (257, 8, 1544, 96, 9, "runs", 0.3), (333, 1288, 8, 88, 1, "one", 0),
    (700, 648, 392, 16, 11, "mixed", 0.2), (1111, 1032, 520, 112, 4, "runs", 0.1), (1500, 264, 264, 56, 1, "one", 0),
    (2100, 136, 1032, 32, 1, "one", 0), (40, 64, 64, 16, 4, "none", 0), (100, 64, 64, 16, 4, "none", 0),
    (5, 64, 64, 8, 300, "mixed", 0), (90, 64, 64, 8, 300, "mixed", 0.2),
    (256, 136, 264, 16, 5, "mixed", 0.1), (400, 64, 72, 8, 300, "mixed", 0.2), (9000, 64, 64, 8, 3, "mixed", 0.1),
    (600, 264, 520, 40, 8, "runs", 0.1), (1100, 264, 520, 64, 1, "one", 0), (1300, 520, 264, 96, 1, "one", 0),
    (1300, 264, 520, 128, 2, "runs", 0.1), (2100, 136, 264, 72, 1, "one", 0), (3, 1544, 2056, 24, 2, "mixed", 0),
    (48, 1032, 6152, 8, 2, "mixed", 0.1), (20, 4104, 1032, 64, 3, "mixed", 0.1), (30, 2056, 1544, 104, 2, "mixed", 0.1),
    (700, 1032, 2056, 40, 12, "mixed", 0.1), (500, 2056, 1032, 16, 40, "runs", 0.1),
    (6, 104, 40, 8, 9, "one", 0), (300, 136, 264, 48, 3, "one", 0), (2100, 136, 136, 40, 2, "one", 0),
    (700, 64, 64, 8, 5000, "mixed", 0.1), (1500, 8, 8, 8, 64, "mixed", 0.1), (700, 8, 8, 8, 4096, "mixed", 0.1),
]
IDS = ["M{}-N{}-K{}-R{}-L{}-{}-{}".format(*c) for c in CASES]


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_forward(case):
    import torch
    note(f"lora forward {case}")
    d = make(*case)
    M, N, K, R = case[:4]
    ref, ref_h = oracle.lora_forward(d["y"], d["x"], d["a"], d["b"], d["index"], d["scaling"])
    # outputs inside larger buffers: rows behind the last stay as they were
    big = torch.full((M + 3, N), 7.0, dtype=torch.float16, device=device())
    big_h = torch.full((M + 3, R), 7.0, device=device())
    out = forward(d, out=big[:M], h=big_h[:M])
    tol, h_tol = forward_tol(d, ref)
    within("h", big_h[:M], ref_h, h_tol)
    within("out", out, ref, tol)
    assert bool((big[M:] == 7).all()) and bool((big_h[M:] == 7).all())
    # the same bits again, without h, and in place
    assert same(forward(d), out)
    y = dev(d["y"])
    w4.w4a16_lora_forward(y, dev(d["x"]), dev(d["a"]), dev(d["b"]), dev(d["index"]), dev(d["scaling"]), out=y)
    assert same(y, out)


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_backward(case):
    note(f"lora backward {case}")
    d = make(*case)
    _, h = oracle.lora_forward(d["y"], d["x"], d["a"], d["b"], d["index"], d["scaling"])
    h = h.astype(np.float32)
    ref = oracle.lora_backward(d["dy"], d["x"], d["a"], d["b"], h, d["index"], d["scaling"], d["dx0"])
    got = backward(d, dev(h))
    for name, g, r, t in zip(("dx", "da", "db"), got, ref, backward_tol(d, h, ref)):
        within(name, g, r, t)
    again = backward(d, dev(h))
    assert all(same(a, b) for a, b in zip(got, again))
    none, da, db = backward(d, dev(h), dx0=False, need_dx=False)
    assert none is None and same(da, got[1]) and same(db, got[2])
    # in place, and without a gradient to add to
    dx = dev(d["dx0"])
    w4.w4a16_lora_backward(dev(d["dy"]), dev(d["x"]), dev(d["a"]), dev(d["b"]), dev(h), dev(d["index"]),
                           dev(d["scaling"]), dx=dx, out=dx)
    assert same(dx, got[0])
    d0 = dict(d, dx0=np.zeros_like(d["dx0"]))
    ref0 = oracle.lora_backward(d["dy"], d["x"], d["a"], d["b"], h, d["index"], d["scaling"])
    within("dx without dx0", backward(d, dev(h), dx0=False)[0], ref0[0], backward_tol(d0, h, ref0)[0])


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("M,N,K,R,L,order", [(1, 64, 128, 8, 1, "one"), (37, 264, 384, 24, 3, "mixed"),
                                             (70, 136, 640, 16, 2, "runs"), (515, 264, 896, 64, 2, "mixed"),
                                             (300, 64, 256, 128, 1, "one")])
def test_backward_from_checkpoint_is_that_of_the_restored_input(M, N, K, R, L, order, group):
    note(f"lora backward q8 {(M, N, K, R, L, order, group)}")
    d = make(M, N, K, R, L, order, 0.1)
    codes, scales = w4.w4a16_act_quantize(dev(d["x"]), group)
    restored = w4.w4a16_act_dequantize(codes, scales, group)
    _, h = oracle.lora_forward(d["y"], d["x"], d["a"], d["b"], d["index"], d["scaling"])
    h = dev(h.astype(np.float32))
    args = (dev(d["a"]), dev(d["b"]), h, dev(d["index"]), dev(d["scaling"]))
    got = w4.w4a16_lora_backward_q8(dev(d["dy"]), codes, scales, group, *args, dx=dev(d["dx0"]))
    want = w4.w4a16_lora_backward(dev(d["dy"]), restored, *args, dx=dev(d["dx0"]))
    assert all(same(a, b) for a, b in zip(got, want))
    x = oracle.act_values(codes.cpu().numpy(), scales.cpu().numpy(), group)
    ref = oracle.lora_backward(d["dy"], x, d["a"], d["b"], h.cpu().numpy(), d["index"], d["scaling"], d["dx0"])
    within("da", got[1], ref[1], backward_tol(dict(d, x=x), h.cpu().numpy(), ref)[1])


@pytest.mark.parametrize("scaling", [True, False])
def test_gradients_match_differences_of_the_forward(scaling):
    """out is linear in A and in B: the change of sum(dy out) under a step D of A is
    sum(dA D), up to the bounds of the two outputs and of the gradient."""
    M, N, K, R, L = 40, 264, 256, 16, 2
    d = make(M, N, K, R, L, "mixed", 0.1, seed=5)
    if not scaling:
        d["scaling"] = None
    import torch
    h = torch.empty((M, R), device=device())
    out0 = forward(d, h=h).double()
    _, da, db = backward(d, h, dx0=False, need_dx=False)
    dy = np.abs(d["dy"].astype(np.float64))
    h32 = h.cpu().numpy()
    _, *tols = backward_tol(d, h32, oracle.lora_backward(d["dy"], d["x"], d["a"], d["b"], h32, d["index"], d["scaling"]))
    tol0 = forward_tol(d, oracle.lora_forward(d["y"], d["x"], d["a"], d["b"], d["index"], d["scaling"])[0])
    for name, grad, grad_tol in (("a", da, tols[0]), ("b", db, tols[1])):
        moved = dict(d, **{name: d[name] * np.float16(-3.0)})
        step = moved[name].astype(np.float64) - d[name].astype(np.float64)
        ref1 = oracle.lora_forward(moved["y"], moved["x"], moved["a"], moved["b"], d["index"], d["scaling"])[0]
        out1 = forward(moved).double()
        change = float((dev(d["dy"]).double() * (out1 - out0)).sum())
        want = float((grad.double().cpu().numpy() * step).sum())
        # h of db carries the forward's own error
        tol = float((dy * (tol0[0] + forward_tol(moved, ref1)[0])).sum()) + float((grad_tol * np.abs(step)).sum())
        if name == "b":
            for i in range(L):
                rows = d["index"] == i
                s = 1.0 if d["scaling"] is None else d["scaling"][i]
                tol += float(s * ((dy[rows].T @ tol0[1][rows]) * np.abs(step[i])).sum())
        assert abs(change - want) <= tol, (name, change, want, tol)


@pytest.mark.parametrize("M", [50, 300])
def test_rows_do_not_touch_each_other(M):
    """NaN and infinities in rows without an adapter, in the rows of another adapter and in
    another adapter's weights stay there; rows without an adapter keep their bits."""
    N, K, R, L = 264, 320, 24, 3
    d = make(M, N, K, R, L, "mixed", 0.2, seed=3)
    clean = {k: (None if v is None else v.copy()) for k, v in d.items()}
    bare, other = d["index"] == -1, d["index"] == 1
    assert bare.any() and other.any()
    d["x"][bare] = np.nan
    d["dy"][bare] = np.inf
    d["x"][other] = np.inf
    d["dy"][other] = np.nan
    d["a"][1] = np.nan
    d["b"][1] = -np.inf
    d["y"][np.nonzero(bare)[0][0]] = np.array(-0.0, np.float16)
    d["y"].view(np.uint16)[np.nonzero(bare)[0][-1]] = 0x7E55            # a NaN with a payload
    keep = ~bare & ~other
    out, ref = forward(d), forward(clean)
    assert same(out[dev(keep)], ref[dev(keep)])
    assert same(out[dev(bare)], dev(d["y"])[dev(bare)])
    _, h = oracle.lora_forward(clean["y"], clean["x"], clean["a"], clean["b"], clean["index"], clean["scaling"])
    h_dirty = h.astype(np.float32)
    h_dirty[bare] = np.nan
    h_dirty[other] = np.inf
    got, want = backward(d, dev(h_dirty)), backward(clean, dev(h.astype(np.float32)))
    assert same(got[0][dev(~other)], want[0][dev(~other)])
    for i in (0, 2):
        assert same(got[1][i], want[1][i]) and same(got[2][i], want[2][i])


def test_adapters_without_rows_get_zero_gradients():
    d = make(300, 64, 64, 16, 4, "last", seed=2)
    d["scaling"][:3] = [np.nan, np.inf, 1.0]
    _, da, db = backward(d, dev(np.ones((300, 16), np.float32)))
    assert not bool(da[:3].any()) and not bool(db[:3].any())
    assert bool(da[3].any()) and bool(da[3].isfinite().all())


def test_non_finite_values_show_in_the_gradients():
    d = make(96, 64, 128, 16, 1, "one")
    d["x"][70, 5] = np.inf
    d["dy"][3, 7] = np.nan
    _, h = oracle.lora_forward(d["y"], make(96, 64, 128, 16, 1, "one")["x"], d["a"], d["b"])
    h[20, 2] = np.inf
    dx, da, db = backward(d, dev(h.astype(np.float32)))
    assert not bool(da.isfinite().all()) and not bool(db.isfinite().all())
    assert bool(dx[3].isnan().all()) and bool(dx[4:].isfinite().all())
    assert bool(da[0, :, 5].isfinite().logical_not().all())
    assert bool(db[0, :, 2].isfinite().logical_not().all())


@pytest.mark.parametrize("x_std,a_std,b_std", [(3000.0, 30.0, 1e-7), (1e-4, 1e-3, 30.0), (1.0, 1e-6, 1.0)])
def test_intermediates_outside_binary16(x_std, a_std, b_std):
    """A x far above the largest binary16, or far below the smallest."""
    d = make(70, 136, 512, 24, 2, "mixed", 0.1, x_std=x_std, a_std=a_std, b_std=b_std)
    d["y"][:] = 0
    ref, ref_h = oracle.lora_forward(d["y"], d["x"], d["a"], d["b"], d["index"], d["scaling"])
    tol, h_tol = forward_tol(d, ref)
    import torch
    h = torch.empty(ref_h.shape, device=device())
    out = forward(d, h=h)
    within("h", h, ref_h, h_tol)
    within("out", out, ref, tol)
    h32 = h.cpu().numpy()
    refs = oracle.lora_backward(d["dy"], d["x"], d["a"], d["b"], h32, d["index"], d["scaling"], d["dx0"])
    tols = backward_tol(d, h32, refs)
    _, da, db = backward(d, h)
    within("da", da, refs[1], tols[1])
    within("db", db, refs[2], tols[2])


def test_rows_of_growing_size_rescale_the_sums():
    """h grows by powers of two from row to row, so the running scale of the outer products
    moves in every chunk; then it falls, so small rows meet a large scale."""
    M, N, K, R = 600, 64, 64, 16
    d = make(M, N, K, R, 1, "one", seed=9)
    _, h = oracle.lora_forward(d["y"], d["x"], d["a"], d["b"])
    for power in (np.arange(M) / 8.0 - 40, 35 - np.arange(M) / 8.0):
        hp = (h * 2.0 ** power[:, None]).astype(np.float32)
        hp[10:20] = 0
        hp[300:340] = 0
        ref = oracle.lora_backward(d["dy"], d["x"], d["a"], d["b"], hp, None, d["scaling"], d["dx0"])
        got = backward(d, dev(hp))
        for name, g, r, t in zip(("dx", "da", "db"), got, ref, backward_tol(d, hp, ref)):
            within(name, g, r, t)


def test_slots_far_below_the_largest_are_not_dropped():
    """256 rows of h of order 1, then 256 rows 2^-k smaller under a dy 2^19 larger: their part
    of the gradient, 2^(19 - k) of the whole, is far above the bound for every k here."""
    N = K = 64
    for k in (18, 22, 24, 25, 26, 28, 30):
        d = make(512, N, K, 16, 1, "one", seed=20 + k)
        _, h = oracle.lora_forward(d["y"], d["x"], d["a"], d["b"])
        h[256:] *= 2.0 ** -k
        d["dy"] = np.concatenate([d["dy"][:256] * np.float16(2.0 ** -9), d["dy"][256:] * np.float16(2.0 ** 10)])
        hp = h.astype(np.float32)
        ref = oracle.lora_backward(d["dy"], d["x"], d["a"], d["b"], hp, None, d["scaling"], d["dx0"])
        got = backward(d, dev(hp))
        within(f"db k={k}", got[2], ref[2], backward_tol(d, hp, ref)[2])


def test_offsets_beyond_32_bits():
    """Adapters and activations of more than 2^31 elements: the last ones count."""
    import torch
    note("lora: 2^31 elements of adapters, then of activations")
    dv = device()
    L, R, K, N = 2080, 128, 8192, 8
    a = torch.zeros((L, R, K), dtype=torch.float16, device=dv)
    b = torch.zeros((L, N, R), dtype=torch.float16, device=dv)
    small = make(3, N, K, R, 1, "one")
    a[L - 1], b[L - 1] = dev(small["a"][0]), dev(small["b"][0])
    index = torch.full((3,), L - 1, dtype=torch.int32, device=dv)
    out = w4.w4a16_lora_forward(dev(small["y"]), dev(small["x"]), a, b, index)
    assert same(out, w4.w4a16_lora_forward(dev(small["y"]), dev(small["x"]), dev(small["a"]), dev(small["b"]),
                                           torch.zeros_like(index)))
    del a, b
    M = 262400
    x = torch.zeros((M, K), dtype=torch.float16, device=dv)
    y = torch.zeros((M, N), dtype=torch.float16, device=dv)
    x[M - 3:], y[M - 3:] = dev(small["x"]), dev(small["y"])
    aa, bb = dev(small["a"]), dev(small["b"])
    out = w4.w4a16_lora_forward(y, x, aa, bb)
    # the batch sizes split the sums differently: compare with the oracle
    ref, _ = oracle.lora_forward(small["y"], small["x"], small["a"], small["b"])
    within("out", out[M - 3:], ref, forward_tol(dict(small, index=None, scaling=None), ref)[0])
    dy = torch.zeros((M, N), dtype=torch.float16, device=dv)
    dy[M - 3:] = dev(small["dy"])
    h = torch.zeros((M, R), device=dv)
    _, h3 = oracle.lora_forward(small["y"], small["x"], small["a"], small["b"])
    h[M - 3:] = dev(h3.astype(np.float32))
    dx, da, db = w4.w4a16_lora_backward(dy, x, aa, bb, h)
    s = dict(small, index=None, scaling=None, dx0=np.zeros_like(small["x"]))
    refs = oracle.lora_backward(small["dy"], small["x"], small["a"], small["b"], h3.astype(np.float32))
    tols = backward_tol(s, h3.astype(np.float32), refs)
    for name, g, r, t in zip(("dx", "da", "db"), (dx[M - 3:], da, db), refs, tols):
        within(name, g, r, t)
    assert not bool(dx[:M - 3].any())


def test_other_stream_and_two_streams_at_once():
    import torch
    d = make(200, 1032, 2056, 32, 3, "mixed", 0.1)
    e = make(180, 1032, 2056, 32, 3, "runs", 0.1, seed=1)
    want = [forward(d), forward(e)]
    args = [[dev(c[k]) for k in ("y", "x", "a", "b", "index", "scaling")] for c in (d, e)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        got = [w4.w4a16_lora_forward(*args[i], stream=streams[i]) for i in (0, 1)]
        torch.cuda.synchronize()
        assert same(got[0], want[0]) and same(got[1], want[1])
    with torch.cuda.stream(streams[0]):
        got = w4.w4a16_lora_forward(*args[0])
    torch.cuda.synchronize()
    assert same(got, want[0])


def test_two_graphs_on_one_stream():
    """Forward, checkpoint and backward captured twice with other inputs; the graphs are
    replayed in turn and on two streams, with eager calls between."""
    import torch
    dv = device()
    s = torch.cuda.Stream(device=dv)

    def step(t):
        h = torch.empty((t["x"].shape[0], t["a"].shape[1]), device=dv)
        out = w4.w4a16_lora_forward(t["y"], t["x"], t["a"], t["b"], t["index"], t["scaling"], h=h)
        codes, scales = w4.w4a16_act_quantize(t["x"], 32)
        return (out, h) + tuple(w4.w4a16_lora_backward_q8(t["dy"], codes, scales, 32, t["a"], t["b"], h, t["index"],
                                                          t["scaling"], dx=t["dx0"]))

    cases = [make(150, 264, 512, 24, 3, "mixed", 0.1, seed=k) for k in range(2)]
    tens = [{k: dev(v) for k, v in c.items()} for c in cases]
    want = [step(t) for t in tens]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for t in tens:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            outs.append(step(t))
        graphs.append(g)
    others = [torch.cuda.Stream(device=dv) for _ in graphs]
    for rep in range(4):
        for o in outs:
            for t in o:
                t.fill_(float("nan"))
        torch.cuda.synchronize()
        for g, st in zip(graphs, others):
            if rep % 2:
                with torch.cuda.stream(st):
                    g.replay()
            else:
                g.replay()
        step(tens[rep % 2])
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert all(same(a, b) for a, b in zip(o, w)), f"replay {rep}"
    # new inputs in the captured buffers
    fresh = make(150, 264, 512, 24, 3, "runs", 0.1, seed=7)
    for k, v in fresh.items():
        tens[0][k].copy_(dev(v))
    graphs[0].replay()
    torch.cuda.synchronize()
    assert all(same(a, b) for a, b in zip(outs[0], step(tens[0])))


def test_refused_on_the_device():
    import torch
    d = make(40, 64, 128, 16, 2, "mixed")
    t = {k: dev(v) for k, v in d.items()}
    with pytest.raises(w4.W4A16Error) as e:
        w4.w4a16_lora_forward(t["y"], t["x"], t["a"][:, :12].contiguous(), t["b"][..., :12].contiguous())
    assert e.value.status == w4.ERR_UNSUPPORTED
    with pytest.raises(w4.W4A16Error) as e:
        w4.w4a16_lora_forward(t["y"][:0], t["x"][:0], t["a"], t["b"])
    assert e.value.status == w4.ERR_INVALID_ARG
    with pytest.raises(ValueError):
        w4.w4a16_lora_forward(t["y"], t["x"], t["a"].cpu(), t["b"]) if torch.cuda.device_count() > 1 else _overlap(t)
    with pytest.raises(TypeError):
        w4.w4a16_lora_forward(t["y"], t["x"], t["a"].cpu(), t["b"])
    with pytest.raises(w4.W4A16Error) as e:        # 2-byte offset: not 16-byte aligned
        flat = torch.zeros(40 * 128 + 1, dtype=torch.float16, device=device())
        w4.w4a16_lora_forward(t["y"], flat[1:].view(40, 128), t["a"], t["b"])
    assert e.value.status == w4.ERR_MISALIGNED


def _overlap(t):
    return w4.w4a16_lora_forward(t["y"], t["x"], t["a"], t["b"], out=t["x"].view(-1)[:40 * 64].view(40, 64))


def test_training_step_around_the_quantised_layer():
    """What a user runs: the 4-bit layer's product, the adapters added to it, the input
    kept in 8 bits; then dy through the restored weights, the adapters' gradients from
    the checkpoint, and the gradient of x in place."""
    import torch
    cfg = wl.custom_config("lora-step", 95, K=1024, N=520, group_size=128, M_list=(96,))
    M, R, L, group = 96, 16, 3, 64
    layer = product_layer(cfg, M)
    d = make(M, cfg.N, cfg.K, R, L, "mixed", 0.1, seed=11)
    d["x"] = layer["x"].cpu().numpy()
    a, b, index, scaling = (dev(d[k]) for k in ("a", "b", "index", "scaling"))
    y = w4.w4a16_gemm(layer["x"], layer["qweight"], layer["scales"], layer["qzeros"], None, cfg.group_size)
    d["y"] = y.cpu().numpy()
    h = torch.empty((M, R), device=device())
    w4.w4a16_lora_forward(y, layer["x"], a, b, index, scaling, out=y, h=h)
    codes, scales = w4.w4a16_act_quantize(layer["x"], group)
    ref, _ = oracle.lora_forward(d["y"], d["x"], d["a"], d["b"], d["index"], d["scaling"])
    within("out", y, ref, forward_tol(d, ref)[0])
    w = w4.w4a16_dequant(layer["qweight"], layer["scales"], layer["qzeros"], None, cfg.group_size, cfg.K)
    dx = dev(d["dy"]) @ w
    d["dx0"] = dx.cpu().numpy()
    dx, da, db = w4.w4a16_lora_backward_q8(dev(d["dy"]), codes, scales, group, a, b, h, index, scaling, dx=dx, out=dx)
    h32 = h.cpu().numpy()
    x8 = oracle.act_values(*oracle.act_quantize(d["x"], group), group)
    refs = oracle.lora_backward(d["dy"], x8, d["a"], d["b"], h32, d["index"], d["scaling"], d["dx0"])
    for name, g, r, t in zip(("dx", "da", "db"), (dx, da, db), refs, backward_tol(dict(d, x=x8), h32, refs)):
        within(name, g, r, t)
