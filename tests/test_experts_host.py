"""The entry points of the mixtures of experts and of the vocabulary head's loss without a
GPU: exported symbols, workspace sizes, and every refusal of the C ABI and the binding
(nothing is launched here: the pointers are made up, and each call is refused before it
would use them)."""

import os
import re

import numpy as np
import pytest
import torch

import w4a16_gemm_amd as w4
from w4a16_gemm_amd import experts, head

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BASE = 1 << 20      # a 16-byte aligned address that is never read


@pytest.mark.parametrize("header,module", [("w4a16_experts.h", experts), ("w4a16_head.h", head)])
def test_library_exports_the_headers(header, module):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", header)).read(), flags=re.S)
    declared = sorted(set(re.findall(r"\b(w[48]a16_\w+)\s*\(", text)))
    assert declared == sorted(module.SIGNATURES)
    for name in declared:
        assert hasattr(w4.lib(), name), name


LAYER = dict(qweight=BASE, scales=BASE, qzeros=BASE, g_idx=None, group=32)
TAIL = dict(workspace=BASE, bytes=1 << 40, stream=None)
ROUTE = dict(logits=BASE, kind=16, M=4, E=8, T=2, renorm=1, index=BASE, weights=BASE, stream=None)
ROUTE_BACK = dict(dweights=BASE, logits=BASE, kind=16, index=BASE, weights=BASE, M=4, E=8, T=2, renorm=1, dlogits=BASE,
                  stream=None)
GEMM = dict(x=BASE, **LAYER, index=BASE, M=700, T=2, E=8, N=64, K=128, y=BASE, **TAIL)
BACK = dict(dy=BASE, **LAYER, index=BASE, dx0=BASE, M=4, T=2, E=8, N=64, K=128, dx=BASE, **TAIL)
LAYER_BACK = dict(dy=BASE, **LAYER, dx0=BASE, M=4, N=64, K=128, dx=BASE, **TAIL)
COMBINE = dict(y=BASE, weights=BASE, M=4, T=2, N=64, out=BASE, stream=None)
COMBINE_BACK = dict(dout=BASE, y=BASE, weights=BASE, M=4, T=2, N=64, dy=BASE, dweights=BASE, stream=None)
LOSS = dict(x=BASE, **LAYER, target=BASE, M=4, N=64, K=128, vocab=60, loss=BASE, lse=BASE, **TAIL)
LOSS_BACK = dict(dloss=BASE, x=BASE, **LAYER, target=BASE, lse=BASE, M=4, N=64, K=128, vocab=60, dx=BASE, **TAIL)

BAD, MIS, UNS = w4.ERR_INVALID_ARG, w4.ERR_MISALIGNED, w4.ERR_UNSUPPORTED
SHAPE = [({"M": 0}, BAD), ({"M": -1}, BAD), ({"N": 0}, BAD), ({"N": -8}, BAD), ({"K": 0}, BAD), ({"N": 60}, BAD),
         ({"K": 96}, UNS), ({"group": 16}, UNS), ({"group": 0}, None), ({"group": 128, "K": 192}, BAD),
         ({"N": (1 << 24) + 16}, UNS), ({"N": 1 << 23, "K": 1024}, UNS), ({"M": (1 << 27) + 1}, UNS),
         ({"workspace": None}, BAD), ({"workspace": BASE + 8}, MIS), ({"bytes": 0}, BAD)]
SLOTS = [({"T": 0}, BAD), ({"T": -2}, BAD), ({"E": 0}, UNS), ({"E": 513}, UNS), ({"M": 1 << 26, "T": 4}, UNS),
         ({"M": 1 << 16, "T": 1 << 16}, UNS)]


def _pointers(wide, narrow=()):
    return ([({n: None}, BAD) for n in (*wide, *narrow)] + [({n: BASE + 8}, MIS) for n in wide]
            + [({n: BASE + 2}, MIS) for n in narrow])


WEIGHTS = ["qweight", "scales"]
ZEROS = [({"qzeros": BASE + 4}, MIS)]
ROUTING = [({"M": 0}, BAD), ({"T": 0}, BAD), ({"T": 9}, BAD), ({"kind": 8}, UNS), ({"E": 0}, UNS), ({"E": 513}, UNS),
           ({"M": (1 << 27) + 1}, UNS), ({"E": 256, "M": (1 << 25) + 1}, UNS)]
COMBINING = [({"M": 0}, BAD), ({"T": 0}, BAD), ({"N": 0}, BAD), ({"N": 12}, BAD), ({"M": 1 << 26, "N": 1024}, UNS),
             ({"M": 1 << 26, "T": 4}, UNS), ({"N": (1 << 24) + 8, "M": 1}, UNS)]
EIGHT = [({"N": 72}, UNS)]
# (name, the accepted call, changes)
CALLS = [
    ("w4a16_route", ROUTE, ROUTING + _pointers([], ["logits", "index", "weights"])),
    ("w4a16_route_backward", ROUTE_BACK,
     ROUTING + _pointers([], ["dweights", "logits", "index", "weights", "dlogits"])),
    ("w4a16_experts_gemm", GEMM, SHAPE + SLOTS + ZEROS + _pointers(["x", "y"] + WEIGHTS, ["index"])
     + [({"M": 1 << 24, "T": 1}, UNS), ({"g_idx": BASE, "K": 64, "M": 1 << 23}, UNS)]),
    ("w8a16_experts_gemm", GEMM, EIGHT + _pointers(["x", "y"] + WEIGHTS, ["index"])),
    ("w4a16_experts_backward", BACK, SHAPE + SLOTS + ZEROS + _pointers(["dy", "dx"] + WEIGHTS, ["index"])
     + [({"dx0": BASE + 8}, MIS), ({"M": 1 << 24}, UNS), ({"M": (1 << 22) + 1, "N": 8, "K": 64}, UNS)]),
    ("w8a16_experts_backward", BACK, EIGHT + _pointers(["dy", "dx"] + WEIGHTS, ["index"])),
    ("w4a16_gemm_backward", LAYER_BACK, SHAPE + ZEROS + _pointers(["dy", "dx"] + WEIGHTS) + [({"dx0": BASE + 8}, MIS)]),
    ("w8a16_gemm_backward", LAYER_BACK, EIGHT + _pointers(["dy", "dx"] + WEIGHTS)),
    ("w4a16_experts_combine", COMBINE, COMBINING + _pointers(["y", "out"], ["weights"])),
    ("w4a16_experts_combine_backward", COMBINE_BACK,
     COMBINING + [({"M": (1 << 23) + 1}, UNS)] + _pointers(["dout", "y", "dy"], ["weights", "dweights"])),
    ("w4a16_head_loss", LOSS, SHAPE + ZEROS + _pointers(["x"] + WEIGHTS, ["target", "loss", "lse"])
     + [({"vocab": 0}, BAD), ({"vocab": 65}, BAD), ({"M": 1 << 24}, UNS)]),
    ("w8a16_head_loss", LOSS, EIGHT + _pointers(["x"] + WEIGHTS, ["target", "loss", "lse"])),
    ("w4a16_head_loss_backward", LOSS_BACK,
     SHAPE + ZEROS + _pointers(["x", "dx"] + WEIGHTS, ["dloss", "target", "lse"]) + [({"vocab": -1}, BAD)]),
    ("w8a16_head_loss_backward", LOSS_BACK, EIGHT + _pointers(["x", "dx"] + WEIGHTS, ["dloss", "target", "lse"])),
]
REFUSED = [(name, good, change, status) for name, good, changes in CALLS for change, status in changes]


@pytest.mark.parametrize("name,good,change,status", REFUSED, ids=[f"{n}-{c}" for n, _, c, _ in REFUSED])
def test_c_abi_refuses(name, good, change, status):
    lib = (head if "head" in name else experts)._lib()
    got = getattr(lib, name)(*dict(good, **change).values())
    assert got == status if status is not None else got != w4.OK
    assert w4.lib().w4a16_last_error()


def test_workspace_sizes():
    lib = experts._lib()
    for fn in (lib.w4a16_experts_gemm_workspace, lib.w4a16_experts_backward_workspace):
        for sizes in [(0, 2, 8, 64, 128), (4, 0, 8, 64, 128), (4, 2, 0, 64, 128), (4, 2, 513, 64, 128), (4, 2, 8, 60, 128),
                      (4, 2, 8, 64, 96), (1 << 26, 4, 8, 64, 128), (1 << 30, 4, 8, 64, 128)]:
            assert fn(*sizes, 0) == 0 and fn(*sizes, 1) == 0, sizes
        assert 0 < fn(700, 2, 8, 64, 128, 0) <= fn(700, 2, 8, 64, 128, 1) + 4096
        assert fn(1 << 24, 2, 8, 8, 64, 1) == 0
    # a token's slots in one launch need no plan, and the rows in stored order under act order
    assert lib.w4a16_experts_gemm_workspace(4, 2, 8, 64, 128, 0) == 0
    assert lib.w4a16_experts_gemm_workspace(4, 2, 8, 64, 128, 1) == 8 * 128 * 2
    # partial sums of every slot: past 32 bits
    assert lib.w4a16_experts_backward_workspace(1 << 18, 2, 8, 64, 8128, 0) > 4 * 8128 << 19
    lib = head._lib()
    for fn in (lib.w4a16_head_loss_workspace, lib.w4a16_head_loss_backward_workspace):
        for sizes in [(0, 64, 128), (4, 60, 128), (4, 64, 96), (1 << 25, 64, 128)]:
            assert fn(*sizes, 0) == 0, sizes
        assert 0 < fn(700, 5008, 128, 0) < fn(700, 5008, 128, 1)
        # bounded by pieces of the rows and of the vocabulary
        assert fn(1 << 19, 151936, 1536, 0) == fn(1 << 15, 151936, 1536, 0) < 1 << 32


# --- the binding ----------------------------------------------------------------------------


def _layer(E=8, N=64, K=128, bits=4, group=32, act=False):
    lib = w4.lib()
    words = getattr(lib, f"w{bits}a16_qweight_words")(N, K, int(act))
    lead = (E,) if E else ()
    return dict(qweight=torch.zeros((*lead, words), dtype=torch.int32),
                scales=torch.zeros((*lead, K // group, N), dtype=torch.float16),
                qzeros=torch.zeros((*lead, K // group, N * bits // 32), dtype=torch.int32),
                g_idx=torch.zeros((*lead, K), dtype=torch.int32) if act else None, group_size=group)


def f16(*shape):
    return torch.zeros(shape, dtype=torch.float16)


def f32(*shape):
    return torch.zeros(shape)


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def _good(name):
    layer = _layer(0 if "head" in name or "gemm_backward" in name else 8)
    return {
        "w4a16_route": dict(logits=f16(4, 8), top_k=2),
        "w4a16_route_backward": dict(dweights=f32(4, 2), logits=f16(4, 8), index=i32(4, 2), weights=f32(4, 2)),
        "w4a16_experts_gemm": dict(x=f16(4, 128), **layer, index=i32(4, 2)),
        "w4a16_experts_backward": dict(dy=f16(4, 2, 64), **layer, index=i32(4, 2), K=128),
        "w4a16_gemm_backward": dict(dy=f16(4, 64), **layer, K=128),
        "w4a16_experts_combine": dict(y=f16(4, 2, 64), weights=f32(4, 2)),
        "w4a16_experts_combine_backward": dict(dout=f16(4, 64), y=f16(4, 2, 64), weights=f32(4, 2)),
        "w4a16_head_loss": dict(x=f16(4, 128), **layer, target=i32(4)),
        "w4a16_head_loss_backward": dict(dloss=f32(4), x=f16(4, 128), **layer, target=i32(4), lse=f32(4)),
    }[name]


NAMES = ["w4a16_route", "w4a16_route_backward", "w4a16_experts_gemm", "w4a16_experts_backward", "w4a16_gemm_backward",
         "w4a16_experts_combine", "w4a16_experts_combine_backward", "w4a16_head_loss", "w4a16_head_loss_backward"]


def _changes(name):
    """One wrong operand at a time: another type, shape, order or nothing at all."""
    for key, value in _good(name).items():
        if not isinstance(value, torch.Tensor):
            continue
        if key != "qzeros":
            yield key, None, "absent"
        yield key, value.to(torch.float64), "type"
        yield key, value.numpy(), "array"
        yield key, value.unsqueeze(0), "dims"
        yield key, torch.cat([value, value], -1), "size"
        yield key, torch.cat([value, value], -1)[..., ::2], "strided"


REFUSALS = [(n, k, v, what) for n in NAMES for k, v, what in _changes(n)
            # a layer's own weight buffer may be longer than the layer, as in the layer's calls
            if not (k == "qweight" and what in ("size", "dims") and ("head" in n or "gemm_backward" in n))]


@pytest.mark.parametrize("name,key,value,what", REFUSALS, ids=[f"{n}-{k}-{w}" for n, k, _, w in REFUSALS])
def test_binding_refuses(name, key, value, what):
    with pytest.raises((TypeError, ValueError)):
        getattr(w4, name)(**dict(_good(name), **{key: value}))


@pytest.mark.parametrize("name", NAMES)
def test_binding_refuses_tensors_of_the_host(name):
    with pytest.raises((TypeError, ValueError, RuntimeError)) as info:
        getattr(w4, name)(**_good(name))
    assert "device" in str(info.value).lower() or "gpu" in str(info.value).lower() or "cuda" in str(info.value).lower()


@pytest.mark.parametrize("change", [dict(group_size=0), dict(group_size=-32), dict(group_size=48), dict(group_size=64)])
def test_binding_refuses_groups_that_do_not_fit(change):
    for name in NAMES:
        if "group_size" in _good(name):
            with pytest.raises((TypeError, ValueError)):
                getattr(w4, name)(**dict(_good(name), **change))
