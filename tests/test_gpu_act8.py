"""Activation checkpoints in 8 bits on the GPU: codes, scales and restored values equal to
the oracle's, bit for bit."""

import numpy as np
import pytest

import oracle
import w4a16_gemm_amd as w4
import workloads as wl
from gpu_common import device, note

pytestmark = pytest.mark.gpu


def check(x, group):
    import torch
    codes, scales = w4.w4a16_act_quantize(torch.from_numpy(x).to(device()), group)
    back = w4.w4a16_act_dequantize(codes, scales, group)
    ref_codes, ref_scales = oracle.act_quantize(x, group)
    ref = oracle.act_values(ref_codes, ref_scales, group)
    s = scales.cpu().numpy()
    nan = np.isnan(ref_scales)
    assert np.array_equal(np.isnan(s), nan)
    assert np.array_equal(s[~nan].view(np.uint16), ref_scales[~nan].view(np.uint16))
    assert np.array_equal(codes.cpu().numpy(), ref_codes)
    b = back.cpu().numpy()
    assert np.array_equal(np.isnan(b), np.isnan(ref))
    assert np.array_equal(b[~np.isnan(ref)], ref[~np.isnan(ref)])


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("M,K", [(1, 128), (1, 1536), (3, 8960), (33, 1536), (513, 384), (2050, 4096)])
def test_matches_the_oracle(M, K, group):
    note(f"act quantize M={M} K={K} g={group}")
    x = wl.activations(wl.custom_config("act8", 940, K=K, N=8, group_size=32, outlier_mult=20.0, M_list=(M,)), M)
    check(x, group)


@pytest.mark.parametrize("group", [32, 64, 128])
def test_special_groups(group):
    rng = np.random.default_rng([92, group])
    rows = [rng.standard_normal(256) * s for s in (1e-8, 6e-8, 1e-6, 1e-4, 1.0, 3e3, 2e4)]
    rows += [np.zeros(256), -np.zeros(256), np.full(256, 65504.0), np.full(256, -65472.0), np.full(256, 2.0 ** -24)]
    with np.errstate(over="ignore"):
        x = np.array(rows).astype(np.float16)
    x[5] = np.where(np.isfinite(x[5]), x[5], 1)
    special = np.ones((4, 256), np.float16)
    special[0, 3] = np.inf
    special[1, 200] = -np.inf
    special[2, 17] = np.nan
    special[3, :] = -np.nan
    check(np.concatenate([x, special]), group)


def test_every_tie_and_neighbour():
    """Groups whose scale is exactly 2^e or an odd 11-bit significand, holding every half
    step of the grid and its neighbours."""
    rng = np.random.default_rng(93)
    rows = []
    for s in np.concatenate([2.0 ** np.arange(-12, 4), rng.integers(1024, 2048, 200) / 1024.0]):
        top = np.float16(127 * s)
        ties = ((np.arange(0, 127) + 0.5) * s).astype(np.float16)
        v = np.concatenate([ties, np.nextafter(ties, np.float16(0)), np.nextafter(ties, np.float16(np.inf)), -ties])
        v = v[np.abs(v.astype(np.float64)) <= float(top)]
        v = np.concatenate([v, np.zeros(-len(v) % 31, np.float16)]).reshape(-1, 31)
        rows.append(np.concatenate([np.full((len(v), 1), top), v], axis=1))
    check(np.concatenate(rows), 32)


def test_every_binary16_magnitude_as_the_largest():
    tops = np.arange(0, 0x7C00, dtype=np.uint16).view(np.float16)
    x = np.zeros((len(tops), 32), np.float16)
    rng = np.random.default_rng(94)
    x[:, 1:] = (tops[:, None].astype(np.float64) * rng.uniform(-1, 1, (len(tops), 31))).astype(np.float16)
    x[:, 0] = tops
    check(x, 32)


def test_given_outputs_streams_and_graph():
    import torch
    dv = device()
    x = torch.randn((130, 256), device=dv).half()
    want = w4.w4a16_act_quantize(x, 64)
    codes = torch.full((133, 256), 9, dtype=torch.uint8, device=dv)
    scales = torch.full((133, 4), 9.0, dtype=torch.float16, device=dv)
    w4.w4a16_act_quantize(x, 64, codes=codes[:130], scales=scales[:130])
    assert torch.equal(codes[:130], want[0]) and torch.equal(scales[:130], want[1])
    assert bool((codes[130:] == 9).all()) and bool((scales[130:] == 9).all())
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = w4.w4a16_act_quantize(x, 64, stream=s)
    back = w4.w4a16_act_dequantize(*got, 64, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(back, w4.w4a16_act_dequantize(*want, 64))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c, sc = w4.w4a16_act_quantize(x, 64)
        r = w4.w4a16_act_dequantize(c, sc, 64)
    for rep in range(3):
        x.copy_(torch.randn((130, 256), device=dv).half())
        g.replay()
        torch.cuda.synchronize()
        now = w4.w4a16_act_quantize(x, 64)
        assert torch.equal(c, now[0]) and torch.equal(sc, now[1]) and torch.equal(r, w4.w4a16_act_dequantize(*now, 64))
    with pytest.raises(ValueError):
        w4.w4a16_act_quantize(x, 64, codes=x.view(torch.uint8).view(-1)[:130 * 256].view(130, 256))


def test_more_than_2_31_values():
    import torch
    dv = device()
    M, K = 262400, 8192
    note("act quantize of 2^31 values")
    x = torch.zeros((M, K), dtype=torch.float16, device=dv)
    tail = wl.random_activations(5, K, 95)
    x[M - 5:] = torch.from_numpy(tail).to(dv)
    codes, scales = w4.w4a16_act_quantize(x, 128)
    back = w4.w4a16_act_dequantize(codes, scales, 128)
    ref = oracle.act_quantize(tail, 128)
    assert np.array_equal(codes[M - 5:].cpu().numpy(), ref[0])
    assert np.array_equal(back[M - 5:].cpu().numpy(), oracle.act_values(*ref, 128))
    assert bool((codes[:5] == 128).all()) and not bool(back[:M - 5].any())
