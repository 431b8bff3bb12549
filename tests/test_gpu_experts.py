"""Mixtures of experts on the GPU against the float64 oracle: products by expert and back
through them, over both widths, odd sizes, ragged, empty and padded groups."""

import numpy as np
import pytest

import oracle
import w4a16_gemm_amd as w4
from experts_common import Layers, backward_tol, dev, f16, gemm_tol, make_index, same, within
from gpu_common import device, note

pytestmark = pytest.mark.gpu

SHAPES = [
    # M, T, E, N, K, bits, group, sym, act, index
    (1, 1, 1, 8, 64, 4, 32, False, False, "distinct"),
    (1, 2, 8, 264, 128, 4, 128, False, False, "distinct"),
    (3, 8, 64, 512, 256, 4, 64, True, False, "distinct"),
    (5, 2, 4, 1000, 320, 4, 32, False, False, "mixed"),
    (17, 3, 5, 72, 1024, 4, 1024, False, False, "mixed"),
    (16, 1, 2, 304, 448, 4, 64, False, True, "distinct"),
    (70, 2, 3, 520, 192, 4, 64, False, False, "skewed"),
    (130, 2, 7, 264, 512, 4, 128, False, True, "mixed"),
    (300, 1, 1, 2056, 256, 4, 128, False, False, "one"),
    (513, 2, 4, 1032, 384, 4, 128, True, False, "skewed"),
    (700, 4, 6, 1288, 128, 4, 64, False, False, "padded"),
    (1000, 1, 2, 5128, 64, 4, 64, False, False, "skewed"),
    (33, 2, 3, 40, 128, 4, 32, False, False, "none"),
    (1, 1, 1, 16, 64, 8, 64, False, False, "distinct"),
    (9, 4, 12, 528, 256, 8, 64, True, False, "distinct"),
    (40, 2, 3, 1040, 320, 8, 32, False, False, "mixed"),
    (129, 1, 2, 272, 512, 8, 512, False, False, "skewed"),
    (257, 2, 3, 2064, 128, 8, 128, False, True, "distinct"),
    (600, 3, 4, 784, 192, 8, 64, False, False, "padded"),
    (1, 4, 16, 1544, 4096, 4, 128, False, False, "distinct"),
    (12, 6, 48, 136, 8960, 4, 128, False, False, "mixed"),
    (2, 2, 3, 4104, 4224, 4, 32, False, True, "distinct"),
    (64, 8, 32, 264, 1536, 4, 64, False, False, "one"),
    (64, 8, 512, 40, 640, 4, 32, True, False, "distinct"),
    (3, 2, 8, 2064, 12352, 8, 64, False, False, "distinct"),
    (20, 4, 8, 528, 4096, 8, 128, True, True, "skewed"),
    # 17 to 64 rows of an expert
    (120, 2, 7, 4104, 192, 4, 32, False, False, "distinct"),
    (90, 2, 4, 6152, 320, 4, 64, True, True, "mixed"),
    (150, 1, 3, 12304, 128, 8, 64, False, False, "distinct"),
    (300, 2, 16, 2064, 256, 8, 128, False, False, "padded"),
]


def case(shape, experts=True):
    M, T, E, N, K, bits, group, sym, act, how = shape
    note(f"experts M={M} T={T} E={E} N={N} K={K} bits={bits} group={group} sym={sym} act={act} {how}")
    rng = np.random.default_rng([93, M, T, E, N, K, bits])
    layers = Layers(E, N, K, bits, group, sym, act)
    return rng, layers, make_index(rng, M, T, E, how)


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_products_by_expert(shape):
    M, T, E, N, K = shape[:5]
    rng, layers, index = case(shape)
    x = f16(rng, (M, K))
    y = layers.fn("experts_gemm")(dev(x), *layers.args, dev(index))
    ref = oracle.experts_gemm(x, layers.W, index)
    within("y", y, ref, gemm_tol(x, layers.W, index, ref))
    again = layers.fn("experts_gemm")(dev(x), *layers.args, dev(index))
    assert same(y, again)


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("add", [False, True], ids=["alone", "added"])
def test_products_back_through_the_experts(shape, add):
    M, T, E, N, K = shape[:5]
    rng, layers, index = case(shape)
    dy = f16(rng, (M, T, N), 0.05)
    dx0 = f16(rng, (M, K), 0.05) if add else None
    run = lambda: layers.fn("experts_backward")(dev(dy), *layers.args, dev(index), K, dx=dev(dx0))   # noqa: E731
    dx = run()
    ref = oracle.experts_backward(dy, layers.W, index, dx0)
    within("dx", dx, ref, backward_tol(dy, layers.W, index, dx0, ref))
    assert same(dx, run())


LAYERS = [(1, 16, 64, 4, 64, False, False), (7, 264, 128, 4, 32, False, False), (64, 1000, 320, 4, 64, True, False),
          (65, 72, 1024, 4, 1024, False, False), (200, 520, 448, 4, 64, False, True), (300, 3080, 256, 4, 128, False, False),
          (1100, 264, 4096, 4, 128, False, False), (2100, 136, 2112, 4, 64, False, False), (5, 272, 128, 8, 64, False, False),
          (300, 1040, 512, 8, 128, True, False), (270, 528, 320, 8, 64, False, True), (1500, 144, 4096, 8, 32, False, False)]


@pytest.mark.parametrize("M,N,K,bits,group,sym,act", LAYERS)
def test_gradient_of_the_layer(M, N, K, bits, group, sym, act):
    note(f"layer backward M={M} N={N} K={K} bits={bits} group={group}")
    rng = np.random.default_rng([94, M, N, K, bits])
    layer = Layers(1, N, K, bits, group, sym, act, experts=False)
    dy, dx0 = f16(rng, (M, N), 0.05), f16(rng, (M, K), 0.05)
    index = np.zeros((M, 1), np.int32)
    ref = oracle.experts_backward(dy[:, None], layer.W, index, dx0)
    out = dev(dx0)
    got = layer.fn("gemm_backward")(dev(dy), *layer.args, K, dx=out, out=out)
    assert got.data_ptr() == out.data_ptr()
    within("dx", got, ref, backward_tol(dy[:, None], layer.W, index, dx0, ref))
