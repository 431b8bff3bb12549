"""Pins of the adapter oracle: the gradients against differences of the forward (which is
linear in x, in A and in B, so a difference quotient has no truncation error), rows without
an adapter, and the 8-bit activations against the symmetric 8-bit weight quantiser and
exact rational arithmetic."""

from fractions import Fraction

import numpy as np
import pytest

import oracle
from exact_ref import fp16_ceil_exact


def _case(M=13, N=24, K=40, R=8, L=3, seed=0):
    rng = np.random.default_rng([77, seed])
    d = {"y": rng.standard_normal((M, N)), "x": rng.standard_normal((M, K)),
         "a": rng.standard_normal((L, R, K)), "b": rng.standard_normal((L, N, R)),
         "index": rng.integers(-1, L, M).astype(np.int32), "scaling": rng.uniform(0.25, 2, L)}
    return d, rng


@pytest.mark.parametrize("with_index", [True, False])
def test_gradients_match_differences(with_index):
    d, rng = _case()
    if not with_index:
        d["index"] = None
    dy = rng.standard_normal(d["y"].shape)
    out, h = oracle.lora_forward(**d)
    dx, da, db = oracle.lora_backward(dy, d["x"], d["a"], d["b"], h, d["index"], d["scaling"])
    base = float((dy * out).sum())
    for name, grad in (("x", dx), ("a", da), ("b", db)):
        step = rng.standard_normal(grad.shape)
        moved = dict(d, **{name: d[name] + step})
        change = float((dy * oracle.lora_forward(**moved)[0]).sum()) - base
        # sums of about 1e4 terms of order 10 in float64
        assert abs(change - float((grad * step).sum())) <= 1e-9 * max(1.0, abs(base), abs(change))


def test_rows_without_adapter_pass_through():
    d, rng = _case()
    d["index"][:5] = [-1, 3, 99, -7, 2 ** 31 - 1]
    out, h = oracle.lora_forward(**d)
    dy = rng.standard_normal(d["y"].shape)
    dx0 = rng.standard_normal(d["x"].shape)
    dx, _, _ = oracle.lora_backward(dy, d["x"], d["a"], d["b"], h, d["index"], d["scaling"], dx0)
    assert np.array_equal(out[:5], d["y"][:5]) and not h[:5].any() and np.array_equal(dx[:5], dx0[:5])


@pytest.mark.parametrize("group", [32, 64, 128])
def test_act_quantize_is_the_symmetric_8bit_scheme(group):
    rng = np.random.default_rng([78, group])
    for scale in (1e-7, 1e-4, 1.0, 300.0):
        x = (rng.standard_normal((9, 256)) * scale).astype(np.float16)
        x[2, :group] = 0
        codes, S = oracle.act_quantize(x, group)
        ref_codes, ref_S = oracle.rtn_quantize_sym(x, group, bits=8)
        assert np.array_equal(codes, ref_codes)
        assert np.array_equal(S.view(np.uint16), ref_S.T.astype(np.float16).copy().view(np.uint16))


def test_act_scale_is_exact_and_restored_values_finite():
    tops = [2.0 ** -24, 3 * 2.0 ** -24, 6.1e-5, 1.0, 126.875, 127.0, 65440.0, 65472.0, 65504.0]
    for top in tops:
        x = np.zeros((1, 32), np.float16)
        x[0, 3] = -top
        x[0, 4] = top / 2
        codes, S = oracle.act_quantize(x, 32)
        exact = fp16_ceil_exact(Fraction(float(x[0, 3])) * -1 / 127)
        assert float(S[0, 0]) == min(float(exact), 515.5)
        back = oracle.act_values(codes, S, 32)
        assert np.isfinite(back).all()
        # half a code step, and the rounding of the product to binary16
        assert abs(float(back[0, 3]) + top) <= float(S[0, 0]) / 2 + 2.0 ** -11 * top + 2.0 ** -25


def test_act_groups_with_nan_or_infinity_restore_nan():
    x = np.ones((2, 128), np.float16)
    x[0, 5] = np.inf
    x[1, 70] = np.nan
    back = oracle.act_values(*oracle.act_quantize(x, 64), 64)
    assert np.isnan(back[0, :64]).all() and np.isfinite(back[0, 64:]).all()
    assert np.isfinite(back[1, :64]).all() and np.isnan(back[1, 64:]).all()
