"""Adapters whose intermediates span far more than one binary16 value holds: every h and g
has to keep its own relative precision, as in fp32, however small it is beside the other
ranks, rows and tiles it is multiplied with.

The bounds are those of test_gpu_lora.py without any term that is relative to the largest
value around: an intermediate enters the second product within 2^-22 of itself."""

import numpy as np
import pytest

import oracle
import w4a16_gemm_amd as w4
from gpu_common import device, note
from test_gpu_lora import U, backward, dev, forward, half_tol, magnitudes, make, same, within

pytestmark = pytest.mark.gpu


def owners(d):
    return np.zeros(len(d["x"]), int) if d["index"] is None else d["index"]


def scalings(d):
    return np.ones(len(d["a"])) if d["scaling"] is None else np.asarray(d["scaling"], np.float64)


def backward_bound(d, h, ref):
    """Tolerances of (dx, da, db)."""
    m = magnitudes(d)
    N, R = d["dy"].shape[1], d["a"].shape[1]
    dx, da, db = np.zeros(m["x"].shape), np.zeros(m["a"].shape), np.zeros(m["b"].shape)
    for i, s in enumerate(scalings(d)):
        rows = np.nonzero(owners(d) == i)[0]
        carried = 2.0 ** -22 + 2 * (2 * max(R, rows.size) + 40) * U
        g = m["dy"][rows] @ m["b"][i]
        g_tol = (2 * N * U + carried) * g
        dx[rows] = s * (g_tol @ m["a"][i])
        da[i] = s * (g_tol.T @ m["x"][rows])
        db[i] = s * carried * (m["dy"][rows].T @ np.abs(h[rows]))
    tiny = 1e-45
    return dx + half_tol(np.abs(ref[0]) + dx) + 2 * U * np.abs(ref[0]), da + tiny, db + tiny


def forward_bound(d, ref):
    m = magnitudes(d)
    K, R = d["x"].shape[1], d["a"].shape[1]
    _, h_mag = oracle.lora_forward(np.zeros_like(m["y"]), m["x"], m["a"], m["b"], d["index"])
    carried = (2 * K * U + 2.0 ** -22 + 2 * (2 * R + 8) * U) * h_mag
    spread = np.zeros_like(m["y"])
    for i, s in enumerate(scalings(d)):
        rows = owners(d) == i
        spread[rows] = s * (carried[rows] @ m["b"][i].T)
    return spread + half_tol(np.abs(ref) + spread) + 2 * U * np.abs(ref)


def check_gradients(d, h):
    h = h.astype(np.float32)
    ref = oracle.lora_backward(d["dy"], d["x"], d["a"], d["b"], h, d["index"], d["scaling"], d["dx0"])
    got = backward(d, dev(h))
    for name, g, r, t in list(zip(("dx", "da", "db"), got, ref, backward_bound(d, h, ref)))[1:]:
        within(name, g, r, t)
    assert all(same(a, b) for a, b in zip(got, backward(d, dev(h))))


# one adapter and several; ranks up to one, two and more blocks; sums in parts; a wavefront
# per 128 channels; rows that do not fill their tile
SHAPES = [(512, 64, 64, 16, 1, "one", 0), (45, 136, 72, 8, 2, "mixed", 0.1), (700, 136, 264, 40, 3, "mixed", 0.1),
          (300, 264, 136, 128, 2, "runs", 0), (2100, 136, 136, 40, 1, "one", 0), (700, 1032, 2056, 40, 12, "mixed", 0.1)]
SHAPE_IDS = ["M{}-N{}-K{}-R{}-L{}-{}-{}".format(*c) for c in SHAPES]


@pytest.mark.parametrize("case", SHAPES, ids=SHAPE_IDS)
def test_gradients_of_ranks_far_apart(case):
    """The ranks of h and of g lie up to 2^30 apart.  They never meet in a gradient."""
    note(f"lora range: ranks {case}")
    d = make(*case, seed=31)
    R = case[3]
    k = np.random.default_rng(R).permutation(np.linspace(0, 30, R).astype(int))
    d["b"] = (np.random.default_rng(32).standard_normal(d["b"].shape) * 2.0 ** (8 - k)).astype(np.float16)
    _, h = oracle.lora_forward(d["y"], d["x"], d["a"], d["b"], d["index"], d["scaling"])
    check_gradients(d, h * 2.0 ** -k)


@pytest.mark.parametrize("where", ["halves", "alternate"])
@pytest.mark.parametrize("case", SHAPES, ids=SHAPE_IDS)
def test_gradients_of_rows_far_apart(case, where):
    """Rows of small h under a large dy, and rows of small g beside a large x: their parts of
    the sums are as large as the others', with the rows in halves or in every tile."""
    M = case[0]
    note(f"lora range: rows {case} {where}")
    for k in (18, 26, 30):
        d = make(*case, seed=33 + k)
        small = np.arange(M) >= M // 2 if where == "halves" else np.arange(M) % 2 == 1
        _, h = oracle.lora_forward(d["y"], d["x"], d["a"], d["b"], d["index"], d["scaling"])
        h[small] *= 2.0 ** -k
        up = np.where(small, 2.0 ** 13, 2.0 ** -13)[:, None]
        d["dy"] = (d["dy"] * up).astype(np.float16)
        d["x"] = (np.clip(d["x"], -4, 4) / up).astype(np.float16)
        check_gradients(d, h)


def test_large_rows_under_a_zero_gradient_leave_no_trace():
    """Rows whose output is not used (dy = 0) may hold any finite h."""
    d = make(300, 64, 72, 24, 1, "one", seed=41)
    _, h = oracle.lora_forward(d["y"], d["x"], d["a"], d["b"], d["index"], d["scaling"])
    for power in (20, 40, 80):
        e = dict(d, dy=d["dy"].copy())
        e["dy"][7::32] = 0
        hp = h.copy()
        hp[7::32] *= 2.0 ** power
        check_gradients(e, hp)


def test_gradients_at_the_ends_of_fp32():
    """Subnormal h, and h near the largest fp32, whose sums still fit."""
    d = make(70, 64, 72, 16, 1, "one", seed=42)
    _, h = oracle.lora_forward(d["y"], d["x"], d["a"], d["b"], d["index"], d["scaling"])
    for power in (-130, -110, 100):
        hp = (h * 2.0 ** power).astype(np.float32)
        ref = oracle.lora_backward(d["dy"], d["x"], d["a"], d["b"], hp, None, d["scaling"], d["dx0"])
        _, _, db = backward(d, dev(hp))
        # below the normal range every product and sum may lose a unit of 2^-149
        within("db", db, ref[2], backward_bound(d, hp, ref)[2] + 2 * 300 * 2.0 ** -149)


@pytest.mark.parametrize("group", [32, 64])
def test_checkpoint_gradients_far_apart(group):
    d = make(500, 136, 320, 40, 2, "mixed", 0.1, seed=43)
    _, h = oracle.lora_forward(d["y"], d["x"], d["a"], d["b"], d["index"], d["scaling"])
    h = (h * 2.0 ** -np.linspace(0, 30, 40).astype(int)).astype(np.float32)
    d["dy"][1::2] *= np.float16(2.0 ** -12)
    d["x"][0::2] *= np.float16(2.0 ** -12)
    codes, scales = w4.w4a16_act_quantize(dev(d["x"]), group)
    x = w4.w4a16_act_dequantize(codes, scales, group)
    args = (dev(d["a"]), dev(d["b"]), dev(h), dev(d["index"]), dev(d["scaling"]))
    got = w4.w4a16_lora_backward_q8(dev(d["dy"]), codes, scales, group, *args, dx=dev(d["dx0"]))
    want = w4.w4a16_lora_backward(dev(d["dy"]), x, *args, dx=dev(d["dx0"]))
    assert all(same(a, b) for a, b in zip(got, want))
    d["x"] = x.cpu().numpy()
    ref = oracle.lora_backward(d["dy"], d["x"], d["a"], d["b"], h, d["index"], d["scaling"], d["dx0"])
    for name, g, r, t in list(zip(("dx", "da", "db"), got, ref, backward_bound(d, h, ref)))[1:]:
        within(name, g, r, t)


def test_many_tiles_of_one_adapter_far_apart():
    """More tiles per wavefront than it remembers one by one: 20 rows, in tiles all over, that
    take the wide path; everything else is zero."""
    d = make(9000, 64, 64, 16, 130, "last", seed=44)
    rows = np.random.default_rng(45).permutation(9000)[:20]
    rest = np.ones(9000, bool)
    rest[rows] = False
    d["dy"][rest] = 0
    _, h = oracle.lora_forward(d["y"], d["x"], d["a"], d["b"], d["index"], d["scaling"])
    h[rows[::2]] *= 2.0 ** 30
    h = h.astype(np.float32)
    few = {k: (v[rows] if k in ("y", "x", "dy", "dx0", "index") else v) for k, v in d.items()}
    ref = oracle.lora_backward(few["dy"], few["x"], d["a"], d["b"], h[rows], few["index"], d["scaling"], few["dx0"])
    got = backward(d, dev(h))
    for name, g, r, t in list(zip(("dx", "da", "db"), got, ref, backward_bound(few, h[rows], ref)))[1:]:
        within(name, g, r, t)


def spread(d, R, first, second, seed):
    """Ranks of `first` [.., R on axis 1 or 2 ..] fall by up to 2^31, those of `second` rise by as
    much: every rank has a like part of the output, from h or g that lie that far apart."""
    k = np.random.default_rng(seed).permutation(np.linspace(0, 31, R).astype(int))
    rng = np.random.default_rng(seed + 1)
    for name, power in ((first, 12 - k), (second, k - 18)):
        along = 2.0 ** (power[:, None] if name == "a" else power[None, :])
        d[name] = (np.clip(rng.standard_normal(d[name].shape), -4, 4) * along).astype(np.float16)


# one launch, two launches, and the stream, each with its ranks; rows of several adapters and
# rows without one
OUTPUTS = [(1, 1536, 1536, 16, 4, "mixed", 0), (9, 520, 776, 32, 2, "mixed", 0), (33, 264, 1024, 48, 5, "runs", 0.2),
           (17, 1000, 8200, 16, 3, "mixed", 0.1), (30, 2056, 2056, 24, 2, "mixed", 0), (20, 4104, 1032, 64, 3, "mixed", 0.1),
           (30, 520, 1544, 96, 1, "one", 0), (65, 264, 1544, 128, 2, "mixed", 0.1),
           (300, 264, 520, 16, 3, "mixed", 0.1), (700, 136, 264, 24, 2, "runs", 0.1), (300, 648, 136, 64, 1, "one", 0),
           (333, 264, 264, 96, 3, "mixed", 0.1), (450, 136, 264, 128, 2, "mixed", 0.1)]
OUTPUT_IDS = ["M{}-N{}-K{}-R{}-L{}-{}-{}".format(*c) for c in OUTPUTS]


@pytest.mark.parametrize("case", OUTPUTS, ids=OUTPUT_IDS)
def test_outputs_of_ranks_far_apart(case):
    import torch
    M, R = case[0], case[3]
    note(f"lora range: out {case}")
    d = make(*case, seed=51)
    d["y"][:] = 0
    spread(d, R, "a", "b", 52)
    d["x"][:M // 2] = 0          # some tiles far apart, some zero
    ref, _ = oracle.lora_forward(d["y"], d["x"], d["a"], d["b"], d["index"], d["scaling"])
    out = forward(d)
    within("out", out, ref, forward_bound(d, ref))
    y, h = dev(d["y"]), torch.empty((M, R), device=device())
    w4.w4a16_lora_forward(y, dev(d["x"]), dev(d["a"]), dev(d["b"]), dev(d["index"]), dev(d["scaling"]), out=y, h=h)
    assert same(y, out)
    # beside a base that is not zero, and only one adapter far apart
    e = make(*case, seed=53)
    e["a"][-1], e["b"][-1] = d["a"][-1], d["b"][-1]
    ref, _ = oracle.lora_forward(e["y"], e["x"], e["a"], e["b"], e["index"], e["scaling"])
    within("out of one adapter", forward(e), ref, forward_bound(e, ref))


@pytest.mark.parametrize("case", [c for c in OUTPUTS if c[2] < 2000] + [(96, 64, 72, 32, 2, "mixed", 0.1)],
                         ids=lambda c: "M{}-N{}-K{}-R{}-L{}-{}-{}".format(*c))
def test_input_gradients_of_ranks_far_apart(case):
    M, R = case[0], case[3]
    note(f"lora range: dx {case}")
    d = make(*case, seed=61)
    spread(d, R, "b", "a", 62)
    d["dy"][M // 2:] = 0
    _, h = oracle.lora_forward(d["y"], d["x"], d["a"], d["b"], d["index"], d["scaling"])
    h = h.astype(np.float32)
    for dx0 in (False, True):
        if not dx0:
            d["dx0"][:] = 0
        else:
            d["dx0"] = make(*case, seed=63)["dx0"]
        ref = oracle.lora_backward(d["dy"], d["x"], d["a"], d["b"], h, d["index"], d["scaling"], d["dx0"])
        got = backward(d, dev(h), dx0=dx0)
        for name, g, r, t in zip(("dx", "da", "db"), got, ref, backward_bound(d, h, ref)):
            within(name, g, r, t)
    dx = dev(d["dx0"])
    w4.w4a16_lora_backward(dev(d["dy"]), dev(d["x"]), dev(d["a"]), dev(d["b"]), dev(h), dev(d["index"]),
                           dev(d["scaling"]), dx=dx, out=dx)
    assert same(dx, got[0])


def floored(d):
    """Operands whose bounds count for subnormal ones.  A matrix instruction aligns its products by
    their operands' exponents, in which every subnormal counts as 2^-14: the steps in which it sums
    are 2^-24 of a product of operands of at least that size."""
    out = dict(d)
    for name in ("x", "a", "b", "dy"):
        v = np.abs(d[name].astype(np.float64))
        out[name] = np.where(v > 0, np.maximum(v, 2.0 ** -14), 0.0)
    return out


@pytest.mark.parametrize("case", [(9, 72, 24, 16, 2, "mixed", 0), (40, 136, 1544, 24, 1, "one", 0), (300, 264, 136, 40, 3, "mixed", 0.1),
                                  (600, 72, 264, 72, 1, "one", 0)], ids=lambda c: "M{}-N{}-K{}-R{}-L{}-{}-{}".format(*c))
def test_subnormal_operands(case):
    """x, A, dy and B around and below 2^-14, down to the smallest binary16."""
    import torch
    note(f"lora range: subnormal {case}")
    d = make(*case, seed=91)
    rng = np.random.default_rng(92)
    for name in ("x", "a", "b", "dy"):
        d[name] = (rng.standard_normal(d[name].shape) * 2.0 ** -rng.integers(13, 24, d[name].shape)).astype(np.float16)
    d["y"][:] = 0
    d["scaling"][:] = 2.0 ** 20
    f = floored(d)
    ref, ref_h = oracle.lora_forward(d["y"], d["x"], d["a"], d["b"], d["index"], d["scaling"])
    h = torch.empty(ref_h.shape, device=device())
    out = forward(d, h=h)
    _, h_mag = oracle.lora_forward(d["y"], f["x"], f["a"], f["b"], d["index"])
    within("h", h, ref_h, 2 * d["x"].shape[1] * U * h_mag + 1e-45)
    within("out", out, ref, forward_bound(f, ref))
    h32 = h.cpu().numpy()
    refs = oracle.lora_backward(d["dy"], d["x"], d["a"], d["b"], h32, d["index"], d["scaling"], d["dx0"])
    for name, g, r, t in zip(("dx", "da", "db"), backward(d, h), refs, backward_bound(f, h32, refs)):
        within(name, g, r, t)
