"""Products by expert where weights or rows are infinite: the formula's infinities, and no NaN
that it does not have."""

import numpy as np
import pytest

import w4a16_gemm_amd as w4
from experts_common import dev
from gpu_common import note

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("K", [64, 192, 320, 1088, 2112, 4160, 4224, 8256])
@pytest.mark.parametrize("M,T", [(1, 1), (5, 2), (40, 2), (300, 2)])
@pytest.mark.parametrize("bits", [4, 8])
def test_infinite_weights(M, T, K, bits):
    """One channel of every second output is beyond binary16: 15 x 6000 in 4 bits, 255 x 400 in 8.
    The others are below 8 x 6000, or 128 x 400, and meet a row of 2^-12: their sums are finite, about K 24000 2^-12."""
    note(f"infinite weights M={M} T={T} K={K} bits={bits}")
    rng = np.random.default_rng([121, M, K, bits])
    E, N = 3, 48
    top, scale = (15, 6000.0) if bits == 4 else (255, 400.0)
    codes = rng.integers(0, top // 2 + 1, (E, N, K)).astype(np.uint8)
    channel = rng.integers(K - 32, K, (E, N))
    for e in range(E):
        for n in range(0, N, 2):
            codes[e, n, channel[e, n]] = top
    pack, zeros = (w4.w4a16_pack, w4.w4a16_pack_zeros) if bits == 4 else (w4.w8a16_pack, w4.w8a16_pack_zeros)
    q = dev(np.stack([pack(codes[e], None, 32) for e in range(E)]))
    s = dev(np.full((E, K // 32, N), scale, np.float16))
    z = dev(np.stack([zeros(np.zeros((K // 32, N), np.uint8)) for _ in range(E)]))
    index = rng.integers(0, E, (M, T)).astype(np.int32)
    x = np.full((M, K), 2.0 ** -12, np.float16)
    gemm = w4.w4a16_experts_gemm if bits == 4 else w4.w8a16_experts_gemm
    y = gemm(dev(x), q, s, z, None, 32, dev(index)).cpu().numpy()
    assert np.isposinf(y[..., ::2]).all()
    # W^ and y are rounded to binary16, half a step of 2^-11 each, and the fp32 sums of 16-bit values are far closer
    ref = (codes.astype(np.float64) * scale)[index].sum(axis=3)[..., 1::2] * 2.0 ** -12
    assert (np.abs(y[..., 1::2] - ref) <= 2.0 ** -9 * ref).all()
