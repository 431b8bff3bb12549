"""Paths of the adapter calls that their size rules choose seldom: gradients from 8-bit
checkpoints summed in parts, with a wavefront per 128 channels, and over a last block of fewer
than 128 channels; the backward pass on other streams and in graphs; refusals on the device."""

import numpy as np
import pytest

import oracle
import w4a16_gemm_amd as w4
from gpu_common import device, note
from test_gpu_lora import backward, dev, make, same, within
from test_gpu_lora_range import backward_bound

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,N,K,R,L,order,bare,group", [
    (70, 136, 160, 16, 2, "mixed", 0.1, 32),          # a last block of 32 channels
    (70, 136, 544, 16, 2, "mixed", 0.1, 32),
    (70, 136, 192, 24, 2, "runs", 0.1, 64),           # of 64
    (2100, 136, 160, 40, 1, "one", 0, 32),            # two parts
    (5000, 136, 192, 16, 1, "one", 0, 64),            # four parts
    (2500, 136, 160, 72, 1, "one", 0, 32),            # two parts, ranks above 64
    (700, 1032, 2080, 40, 12, "mixed", 0.1, 32),      # a wavefront per 128 channels
    (500, 2056, 1088, 16, 40, "runs", 0.1, 64),
    (600, 1032, 2080, 104, 8, "mixed", 0.1, 32)])
def test_checkpoint_gradients(M, N, K, R, L, order, bare, group):
    note(f"lora paths q8 {(M, N, K, R, L, order, group)}")
    d = make(M, N, K, R, L, order, bare, seed=71)
    codes, scales = w4.w4a16_act_quantize(dev(d["x"]), group)
    restored = w4.w4a16_act_dequantize(codes, scales, group)
    _, h = oracle.lora_forward(d["y"], d["x"], d["a"], d["b"], d["index"], d["scaling"])
    h = h.astype(np.float32)
    args = (dev(d["a"]), dev(d["b"]), dev(h), dev(d["index"]), dev(d["scaling"]))
    got = w4.w4a16_lora_backward_q8(dev(d["dy"]), codes, scales, group, *args, dx=dev(d["dx0"]))
    want = w4.w4a16_lora_backward(dev(d["dy"]), restored, *args, dx=dev(d["dx0"]))
    assert all(same(a, b) for a, b in zip(got, want))
    d["x"] = oracle.act_values(codes.cpu().numpy(), scales.cpu().numpy(), group)
    ref = oracle.lora_backward(d["dy"], d["x"], d["a"], d["b"], h, d["index"], d["scaling"], d["dx0"])
    for name, g, r, t in zip(("dx", "da", "db"), got, ref, backward_bound(d, h, ref)):
        within(name, g, r, t)
    none, da, db = w4.w4a16_lora_backward_q8(dev(d["dy"]), codes, scales, group, *args, need_dx=False)
    assert none is None and same(da, got[1]) and same(db, got[2])


def _wide(seed, M=300):
    """A step whose rows and ranks lie far apart, and its h."""
    d = make(M, 264, 520, 40, 3, "mixed", 0.1, seed=seed)
    d["dy"][1::2] *= np.float16(2.0 ** -12)
    d["x"][0::2] *= np.float16(2.0 ** -12)
    d["a"] = (d["a"] * 2.0 ** (8 - np.linspace(0, 20, 40).astype(int))[:, None]).astype(np.float16)
    _, h = oracle.lora_forward(d["y"], d["x"], d["a"], d["b"], d["index"], d["scaling"])
    return d, h.astype(np.float32)


def test_backward_on_two_streams_at_once():
    import torch
    both = [_wide(81), _wide(82, 310)]
    want = [backward(d, dev(h)) for d, h in both]
    args = [[dev(d[k]) for k in ("dy", "x", "a", "b")] + [dev(h), dev(d["index"]), dev(d["scaling"])] for d, h in both]
    dx0 = [dev(d["dx0"]) for d, _ in both]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        got = [w4.w4a16_lora_backward(*args[i], dx=dx0[i], stream=streams[i]) for i in (0, 1)]
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert all(same(a, b) for a, b in zip(g, w))


@pytest.mark.parametrize("M", [40, 300])
def test_graph_of_a_step_far_apart(M):
    """Forward and backward captured; replayed with eager calls and other inputs between."""
    import torch
    dv = device()
    d, _ = _wide(83, M)
    t = {k: dev(v) for k, v in d.items()}

    def step(t):
        h = torch.empty((M, 40), device=dv)
        out = w4.w4a16_lora_forward(t["y"], t["x"], t["a"], t["b"], t["index"], t["scaling"], h=h)
        plain = w4.w4a16_lora_forward(t["y"], t["x"], t["a"], t["b"], t["index"], t["scaling"])
        return (out, plain, h) + tuple(w4.w4a16_lora_backward(t["dy"], t["x"], t["a"], t["b"], h, t["index"],
                                                              t["scaling"], dx=t["dx0"]))

    want = step(t)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = step(t)
    for seed in (83, 84, 83, 85):
        fresh, _ = _wide(seed, M)
        for k, v in fresh.items():
            t[k].copy_(dev(v))
        for o in outs:
            o.fill_(float("nan"))
        torch.cuda.synchronize()
        g.replay()
        want = step(t)
        torch.cuda.synchronize()
        assert all(same(a, b) for a, b in zip(outs, want)), f"seed {seed}"
        assert same(outs[0], outs[1])


def test_refusals_on_the_device():
    import torch
    M, N, K, R = 40, 64, 128, 16
    d = make(M, N, K, R, 2, "mixed")
    t = {k: dev(v) for k, v in d.items()}
    h = torch.zeros((M, R), device=device())
    fwd = (t["y"], t["x"], t["a"], t["b"], t["index"], t["scaling"])
    bwd = (t["dy"], t["x"], t["a"], t["b"], h, t["index"], t["scaling"])
    with pytest.raises(ValueError, match="overlaps x"):
        w4.w4a16_lora_forward(*fwd, out=t["x"].view(-1)[:M * N].view(M, N))
    with pytest.raises(ValueError, match="overlaps x"):
        w4.w4a16_lora_forward(*fwd, h=t["x"].view(torch.float32).view(-1)[:M * R].view(M, R))
    both = torch.zeros((M + 1, N), dtype=torch.float16, device=device())
    with pytest.raises(ValueError, match="overlaps y"):     # in place, but a row further
        w4.w4a16_lora_forward(both[:M], *fwd[1:], out=both[1:])
    out = torch.zeros((M, N), dtype=torch.float16, device=device())
    with pytest.raises(ValueError, match="overlaps h"):
        w4.w4a16_lora_forward(*fwd, out=out, h=out.view(torch.float32).view(-1)[:M * R].view(M, R))
    wide = torch.zeros((M, K), dtype=torch.float16, device=device())
    with pytest.raises(ValueError, match="overlaps dy"):
        w4.w4a16_lora_backward(wide.view(-1)[:M * N].view(M, N), *bwd[1:], out=wide)
    rows = torch.zeros((M + 1, K), dtype=torch.float16, device=device())
    with pytest.raises(ValueError, match="overlaps dx"):
        w4.w4a16_lora_backward(*bwd, dx=rows[:M], out=rows[1:])
    with pytest.raises(ValueError, match="need_dx"):
        w4.w4a16_lora_backward(*bwd, dx=t["dx0"], need_dx=False)
    with pytest.raises(ValueError, match="need_dx"):
        w4.w4a16_lora_backward(*bwd, out=t["dx0"], need_dx=False)
    codes, scales = w4.w4a16_act_quantize(t["x"], 32)
    room = torch.zeros((M, K), dtype=torch.float16, device=device())
    inside = room.view(torch.uint8).view(-1)[:M * K].view(M, K)
    with pytest.raises(ValueError, match="overlaps codes"):
        w4.w4a16_lora_backward_q8(t["dy"], inside, scales, 32, *bwd[2:], out=room)
    with pytest.raises(w4.W4A16Error) as e:
        w4.w4a16_lora_backward_q8(t["dy"], codes, torch.zeros((M, 2), dtype=torch.float16, device=device()), 48, *bwd[2:])
    assert e.value.status == w4.ERR_UNSUPPORTED
    for name in ("dy", "x", "a", "b"):
        at = ("dy", "x", "a", "b").index(name)
        with pytest.raises(TypeError):
            w4.w4a16_lora_backward(*bwd[:at], bwd[at].cpu(), *bwd[at + 1:])


@pytest.mark.parametrize("M,K,R", [(14, 64, 16), (14, 64, 24), (14, 6152, 16), (30, 1544, 64), (30, 1544, 96), (300, 64, 16),
                                   (300, 64, 32), (300, 64, 48), (300, 64, 72), (300, 64, 128)])
def test_a_row_does_not_depend_on_rows_far_apart(M, K, R):
    """Ranks 0 .. R - 2 read one half of the channels, the last rank the other half.  Every third
    row has a tiny second half, so that its ranks lie 2^24 apart: the others keep their bits, in out
    and (with the roles of A and B exchanged) in dx."""
    import torch
    N = 136
    d = make(M, N, K, R, 1, "one", seed=77)
    d["a"][0, :-1, K // 2:] = 0
    d["a"][0, -1, :K // 2] = 0
    far = np.arange(M) % 3 == 1
    e = dict(d, x=d["x"].copy())
    e["x"][far, :K // 2] *= np.float16(2.0 ** 10)
    e["x"][far, K // 2:] *= np.float16(2.0 ** -14)
    plain, other = w4.w4a16_lora_forward, {}
    for name, c in (("d", d), ("e", e)):
        h = torch.empty((M, R), device=device())
        other[name] = (plain(dev(c["y"]), dev(c["x"]), dev(c["a"]), dev(c["b"]), None, dev(c["scaling"]), h=h), h)
    assert same(other["d"][0][dev(~far)], other["e"][0][dev(~far)])
    assert same(other["d"][1][dev(~far)], other["e"][1][dev(~far)])
    h = np.abs(other["e"][1].cpu().numpy())
    assert np.median(h[far, :-1].max(axis=1) / h[far, -1]) > 2.0 ** 20      # far apart indeed
    # dx: the first half of dy's channels reaches all ranks but the last
    d["b"] = np.zeros((1, N, R), np.float16)
    d["b"][0, :N // 2, :-1] = make(1, N // 2, 8, R, 1, "one", seed=78)["b"][0][:, :-1]
    d["b"][0, N // 2:, -1] = 0.5
    e = dict(d, dy=d["dy"].copy())
    e["dy"][far, :N // 2] *= np.float16(2.0 ** 10)
    e["dy"][far, N // 2:] *= np.float16(2.0 ** -10)
    h0 = torch.zeros((M, R), device=device())
    got = [w4.w4a16_lora_backward(dev(c["dy"]), dev(c["x"]), dev(c["a"]), dev(c["b"]), h0, None, dev(c["scaling"]),
                                  dx=dev(c["dx0"]))[0] for c in (d, e)]
    assert same(got[0][dev(~far)], got[1][dev(~far)])
