"""Inputs, bounds and comparisons shared by the GPU tests of the mixtures of experts and of
the vocabulary head's loss.

Bounds, not fits.  u = 2^-24.  An fp32 sum of n products in any order is within 2 n u of
sum |p|, the factor 2 for matrix instructions that add several products with truncation;
there an operand below 2^-14 counts as 2^-14.  A binary16 result adds half a step, 2^-11 of
itself, and half a subnormal step, 2^-25."""

import numpy as np

import oracle
import w4a16_gemm_amd as w4
from gpu_common import device

U = 2.0 ** -24


def dev(a):
    import torch
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(device())


def bits(t):
    import torch
    return t.contiguous().view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[t.element_size()])


def same(a, b):
    import torch
    return torch.equal(bits(a), bits(b))


def half_tol(ref):
    return 2.0 ** -11 * np.abs(ref) + 2.0 ** -25


def floored(a):
    """|a| as it counts in the errors of a matrix instruction's sums."""
    return np.maximum(np.abs(np.asarray(a, np.float64)), 2.0 ** -14)


def within(name, got, ref, tol):
    got = got.detach().cpu().numpy().astype(np.float64)
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    err = np.abs(got - ref)
    bad = ~(err <= tol)
    assert not bad.any(), (f"{name}: {int(bad.sum())} of {bad.size} beyond the bound, worst "
                           f"{np.nanmax(np.where(bad, err / tol, 0)):.3g} times it, first at "
                           f"{np.unravel_index(np.argmax(bad), bad.shape)}: {got[bad][0]} for {ref[bad][0]}")


class Layers:
    """E packed layers of random codes (one without a leading size: experts=False)."""

    def __init__(self, E, N, K, bits=4, group=128, sym=False, act=False, seed=0, experts=True, scale=0.004):
        rng = np.random.default_rng([92, E, N, K, bits, group, int(sym), int(act), seed])
        self.E, self.N, self.K, self.bits, self.group = E, N, K, bits, group
        G = K // group
        top = 1 << bits
        four = bits == 4
        spread = 16 // top if four else 16 / top
        self.codes = rng.integers(0, top, (E, N, K), dtype=np.int64).astype(np.uint8)
        self.S = (rng.uniform(0.5, 1.5, (E, G, N)) * scale * spread).astype(np.float16)
        self.Z = np.full((E, G, N), top // 2) if sym else rng.integers(top // 4, 3 * top // 4, (E, G, N))
        self.Z = self.Z.astype(np.uint8)
        self.g_idx = None
        if act:
            self.g_idx = np.stack([rng.permutation(np.repeat(np.arange(G), group)) for _ in range(E)]).astype(np.int32)
        gi = (lambda e: None if self.g_idx is None else self.g_idx[e])
        pack, pack_zeros = (w4.w4a16_pack, w4.w4a16_pack_zeros) if four else (w4.w8a16_pack, w4.w8a16_pack_zeros)
        self.W = np.stack([oracle.dequant_fp16(self.codes[e], self.S[e], self.Z[e], group, gi(e)) for e in range(E)])
        q = np.stack([pack(self.codes[e], gi(e), group) for e in range(E)])
        z = None if sym else np.stack([pack_zeros(self.Z[e]) for e in range(E)])
        cut = (lambda a: a if experts or a is None else a[0])
        self.args = (dev(cut(q)), dev(cut(self.S)), dev(cut(z)), dev(cut(self.g_idx)), group)

    def fn(self, name):
        return getattr(w4, f"w{self.bits}a16_{name}")


def make_index(rng, M, T, E, how):
    if how == "distinct":
        index = np.argsort(rng.random((M, E)), axis=1)[:, :T]
    elif how == "mixed":                          # experts may repeat within a row
        index = rng.integers(0, E, (M, T))
        index[rng.random((M, T)) < 0.2] = -1
    elif how == "one":
        index = np.full((M, T), E - 1)
    elif how == "none":
        index = rng.choice([-1, E, -2 ** 31, 2 ** 31 - 1], (M, T))
    elif how == "skewed":                         # one expert has most of the rows, some have none
        index = np.where(rng.random((M, T)) < 0.85, 0, rng.integers(0, max(1, E // 2), (M, T)))
    elif how == "padded":
        index = np.argsort(rng.random((M, E)), axis=1)[:, :T]
        index[M // 2:] = -1
    else:
        raise ValueError(how)
    return index.astype(np.int32)


def f16(rng, shape, std=1.0):
    return (rng.standard_normal(shape) * std).astype(np.float16)


def gemm_tol(x, W, index, ref):
    K = x.shape[1]
    mag = oracle.experts_gemm(floored(x), floored(W), index)
    return 2 * K * U * mag + half_tol(ref) + 2 * U * np.abs(ref)


def backward_tol(dy, W, index, dx0, ref):
    """A partial sum per slot and part, then up to 16 parts of T slots and dx0."""
    M, T, N = dy.shape
    mag = oracle.experts_backward(floored(dy), floored(W), index)
    if dx0 is not None:
        mag = mag + np.abs(dx0.astype(np.float64))
    return (2 * N + 16 * T + 2) * U * mag + half_tol(ref)
