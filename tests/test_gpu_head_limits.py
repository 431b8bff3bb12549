"""The vocabulary head's loss at the edges of what one launch takes."""

import numpy as np
import pytest

import w4a16_gemm_amd as w4
from experts_common import U, Layers, dev, f16, within
from gpu_common import device, note
from test_gpu_head import loss_tol

pytestmark = pytest.mark.gpu


def test_loss_of_more_rows_and_outputs_than_one_launch_takes():
    """33000 rows against 2^24 outputs: 2^32 threads and more in one launch of 256-row tiles.  The
    head is one of 4096 outputs over and over, each time with scales of its own, powers of two from
    2^-10 to 2^-6, so that W^ is exact and a logit is its output's scale times one of 4096 sums."""
    import torch
    note("loss of 33000 rows against 2^24 outputs")
    rng = np.random.default_rng(120)
    M, K, base, N = 33000, 64, 4096, 1 << 24
    vocab = N - 3
    layer = Layers(1, base, K, 4, 64, experts=False)
    q, _, z, _, group = layer.args
    times = N // base
    q, z = q.repeat(times), z.repeat(1, times)
    exponent = torch.randint(-10, -5, (1, N), generator=torch.Generator(device="cuda").manual_seed(3), device=device())
    scales = torch.pow(2.0, exponent.double()).half()
    x, target = f16(rng, (M, K)), rng.integers(0, vocab, M).astype(np.int32)
    target[::11] = -100
    loss, lse = w4.w4a16_head_loss(dev(x), q, scales, z, None, group, dev(target), vocab=vocab)
    torch.cuda.synchronize()
    rows = np.r_[0:3, 4030:4034, 16000, 32766:32770, M - 3:M]
    signs = layer.codes[0].astype(np.float64) - np.repeat(layer.Z[0].T.astype(np.float64), K, 1)
    sums = dev(x[rows].astype(np.float64) @ signs.T)
    ref_lse, ref_loss = np.zeros(len(rows)), np.zeros(len(rows))
    for i, m in enumerate(rows):
        if target[m] < 0:
            continue
        l = (sums[i].repeat(times) * scales[0].double())[:vocab]
        ref_lse[i] = torch.logsumexp(l, 0).item()
        ref_loss[i] = ref_lse[i] - l[int(target[m])].item()
    tol = loss_tol(x[rows], signs * 2.0 ** -6, ref_lse)
    more = N / 2048 * U                     # its sums are over N outputs
    within("lse", lse[dev(rows)], ref_lse, tol[1] + more)
    within("loss", loss[dev(rows)], ref_loss, tol[0] + more)
    none = dev(target < 0)
    assert not loss[none].any() and not lse[none].any()
    assert torch.isfinite(loss).all() and (lse[~none] > 0).all()
