"""The adapter entry points without a GPU: exported symbols, workspace sizes, and every
refusal of the C ABI and the binding (nothing is launched here: the pointers are made up,
and each call is refused before it would use them)."""

import ctypes
import os
import re

import numpy as np
import pytest
import torch

import w4a16_gemm_amd as w4
from w4a16_gemm_amd import adapters

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BASE = 1 << 20      # a 16-byte aligned address that is never read


def test_library_exports_the_adapter_header():
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "w4a16_adapters.h")).read(), flags=re.S)
    declared = sorted(set(re.findall(r"\b(w4a16_\w+)\s*\(", text)))
    assert declared == sorted(adapters.SIGNATURES)
    for name in declared:
        assert hasattr(w4.lib(), name), name


FORWARD = dict(y=BASE, x=BASE, a=BASE, b=BASE, index=BASE, scaling=BASE, M=4, N=64, K=8192, R=16, L=2, out=BASE, h=BASE,
               workspace=BASE, bytes=1 << 30, stream=None)
BACKWARD = dict(dy=BASE, x=BASE, a=BASE, b=BASE, h=BASE, index=BASE, scaling=BASE, dx0=BASE, M=4, N=64, K=128, R=16, L=2,
                dx=BASE, da=BASE, db=BASE, workspace=BASE, bytes=1 << 30, stream=None)
Q8 = dict(dy=BASE, codes=BASE, scales=BASE, group=32, a=BASE, b=BASE, h=BASE, index=BASE, scaling=BASE, dx0=BASE, M=4,
          N=64, K=128, R=16, L=2, dx=BASE, da=BASE, db=BASE, workspace=BASE, bytes=1 << 30, stream=None)
QUANT = dict(x=BASE, M=4, K=128, group=32, codes=BASE, scales=BASE, stream=None)
DEQUANT = dict(codes=BASE, scales=BASE, M=4, K=128, group=32, x=BASE, stream=None)

SHAPE = [({"M": 0}, w4.ERR_INVALID_ARG), ({"M": -1}, w4.ERR_INVALID_ARG), ({"N": 0}, w4.ERR_INVALID_ARG),
         ({"K": 0}, w4.ERR_INVALID_ARG), ({"N": 60}, w4.ERR_INVALID_ARG), ({"K": 100}, w4.ERR_INVALID_ARG),
         ({"R": 0}, w4.ERR_UNSUPPORTED), ({"R": 12}, w4.ERR_UNSUPPORTED), ({"R": 136}, w4.ERR_UNSUPPORTED),
         ({"L": 0}, w4.ERR_UNSUPPORTED), ({"L": 65536}, w4.ERR_UNSUPPORTED), ({"M": (1 << 27) + 1}, w4.ERR_UNSUPPORTED),
         ({"N": (1 << 24) + 8}, w4.ERR_UNSUPPORTED), ({"bytes": 16}, w4.ERR_INVALID_ARG),
         ({"workspace": None}, w4.ERR_INVALID_ARG), ({"workspace": BASE + 8}, w4.ERR_MISALIGNED)]
GROUP = [({"group": 16}, w4.ERR_UNSUPPORTED), ({"group": 0}, w4.ERR_UNSUPPORTED), ({"group": 128, "K": 192}, w4.ERR_INVALID_ARG),
         ({"codes": None}, w4.ERR_INVALID_ARG), ({"scales": None}, w4.ERR_INVALID_ARG),
         ({"codes": BASE + 4}, w4.ERR_MISALIGNED), ({"scales": BASE + 1}, w4.ERR_MISALIGNED)]


def _pointers(names):
    return [({n: None}, w4.ERR_INVALID_ARG) for n in names] + [({n: BASE + 2}, w4.ERR_MISALIGNED) for n in names]


REFUSED = (
    [("w4a16_lora_forward", FORWARD, c) for c in SHAPE + _pointers(["y", "x", "a", "b", "out"])
     + [({"index": BASE + 2}, w4.ERR_MISALIGNED), ({"scaling": BASE + 2}, w4.ERR_MISALIGNED), ({"h": BASE + 4}, w4.ERR_MISALIGNED)]]
    + [("w4a16_lora_backward", BACKWARD, c) for c in SHAPE + _pointers(["dy", "x", "a", "b", "h", "da", "db"])
       + [({"dx": None}, w4.ERR_INVALID_ARG), ({"dx0": BASE + 2}, w4.ERR_MISALIGNED)]]
    + [("w4a16_lora_backward_q8", Q8, c) for c in SHAPE + GROUP + _pointers(["dy", "a", "b", "h", "da", "db"])]
    + [("w4a16_act_quantize", QUANT, c) for c in GROUP + _pointers(["x"]) + [({"M": 0}, w4.ERR_INVALID_ARG), ({"K": -32}, w4.ERR_INVALID_ARG), ({"M": 1 << 30}, w4.ERR_UNSUPPORTED)]]
    + [("w4a16_act_dequantize", DEQUANT, c) for c in GROUP + _pointers(["x"]) + [({"M": 0}, w4.ERR_INVALID_ARG), ({"M": 1 << 30}, w4.ERR_UNSUPPORTED)]])


@pytest.mark.parametrize("name,good,change", REFUSED, ids=[f"{n}-{c[0]}" for n, _, c in REFUSED])
def test_c_abi_refuses(name, good, change):
    args, status = change
    fn = getattr(adapters._lib(), name)
    assert fn(*dict(good, **args).values()) == status
    assert w4.lib().w4a16_last_error()


def test_workspace_sizes():
    lib = adapters._lib()
    for fn in (lib.w4a16_lora_forward_workspace, lib.w4a16_lora_backward_workspace):
        assert fn(4, 64, 128, 12, 2, 1) == 0 and fn(0, 64, 128, 16, 2, 1) == 0
        assert 0 < fn(4, 64, 8192, 16, 2, 0) <= fn(4, 64, 8192, 16, 2, 1)
        assert fn(1000, 64, 128, 16, 2, 1) >= fn(1000, 64, 128, 16, 2, 0) + 4 * 1002
    # few rows of a small layer need none, and take a NULL workspace
    assert lib.w4a16_lora_forward_workspace(4, 64, 128, 16, 2, 1) == 0
    # sizes that pass 32 bits
    assert lib.w4a16_lora_backward_workspace(1 << 24, 64, 128, 128, 2, 0) >= 4 * 128 << 24


# --- the binding ---------------------------------------------------------------------

def _tensors():
    t = torch.zeros
    return dict(y=t(4, 64, dtype=torch.float16), x=t(4, 128, dtype=torch.float16),
                a=t(2, 16, 128, dtype=torch.float16), b=t(2, 64, 16, dtype=torch.float16),
                index=t(4, dtype=torch.int32), scaling=t(2), out=t(4, 64, dtype=torch.float16), h=t(4, 16))


@pytest.mark.parametrize("change", [
    {"y": torch.zeros(5, 64, dtype=torch.float16)}, {"x": torch.zeros(4, 120, dtype=torch.float16)},
    {"b": torch.zeros(2, 16, 64, dtype=torch.float16)}, {"b": torch.zeros(3, 64, 16, dtype=torch.float16)},
    {"a": torch.zeros(16, 128, dtype=torch.float16)}, {"index": torch.zeros(3, dtype=torch.int32)},
    {"scaling": torch.zeros(3)}, {"out": torch.zeros(4, 56, dtype=torch.float16)}, {"h": torch.zeros(4, 8)},
    {"x": torch.zeros(128, dtype=torch.float16)}])
def test_forward_refuses_shapes(change):
    with pytest.raises(ValueError):
        w4.w4a16_lora_forward(**dict(_tensors(), **change))


@pytest.mark.parametrize("change", [
    {"y": torch.zeros(4, 64)}, {"x": torch.zeros(4, 128, dtype=torch.bfloat16)}, {"index": torch.zeros(4, dtype=torch.int64)},
    {"scaling": torch.zeros(2, dtype=torch.float64)}, {"h": torch.zeros(4, 16, dtype=torch.float16)},
    {"x": torch.zeros(128, 4, dtype=torch.float16).t()}, {}])
def test_forward_refuses_types_layouts_and_host_tensors(change):
    with pytest.raises(TypeError):
        w4.w4a16_lora_forward(**dict(_tensors(), **change))


def _backward_tensors():
    d = _tensors()
    return dict(dy=d["y"], x=d["x"], a=d["a"], b=d["b"], h=d["h"], index=d["index"], scaling=d["scaling"],
                dx=torch.zeros(4, 128, dtype=torch.float16))


@pytest.mark.parametrize("change,error", [
    ({"dy": torch.zeros(3, 64, dtype=torch.float16)}, ValueError), ({"h": torch.zeros(4, 8)}, ValueError),
    ({"h": None}, TypeError), ({"dx": torch.zeros(4, 64, dtype=torch.float16)}, ValueError), ({}, TypeError)])
def test_backward_refuses(change, error):
    with pytest.raises(error):
        w4.w4a16_lora_backward(**dict(_backward_tensors(), **change))


def test_checkpoint_calls_refuse():
    codes, scales = torch.zeros(4, 128, dtype=torch.uint8), torch.zeros(4, 4, dtype=torch.float16)
    d = _backward_tensors()
    rest = (d["a"], d["b"], d["h"])
    with pytest.raises(ValueError):
        w4.w4a16_lora_backward_q8(d["dy"], codes, scales, 64, *rest)          # scales of another group size
    with pytest.raises(TypeError):
        w4.w4a16_lora_backward_q8(d["dy"], codes.to(torch.int8), scales, 32, *rest)
    with pytest.raises(TypeError):
        w4.w4a16_lora_backward_q8(d["dy"], codes, None, 32, *rest)
    with pytest.raises(TypeError):
        w4.w4a16_lora_backward_q8(d["dy"], codes, scales, 32, *rest)          # host tensors
    with pytest.raises(TypeError):
        w4.w4a16_act_quantize(d["x"], 32)
    with pytest.raises(ValueError):
        w4.w4a16_act_dequantize(codes, scales, 128)
    with pytest.raises(ValueError):
        w4.w4a16_act_dequantize(codes[0], scales, 32)


def test_overlapping_outputs_are_found():
    x = torch.zeros(8, 64, dtype=torch.float16)
    adapters._overlap(x[:4], (x[4:], "x"))
    with pytest.raises(ValueError):
        adapters._overlap(x[:5], (x[4:], "x"))


def test_sizes_beyond_the_int_arguments_are_refused():
    big = lambda *shape, dtype=torch.float16: torch.empty(*shape, dtype=dtype, device="meta")   # noqa: E731
    rows = 2 ** 32 + 4      # 4 rows, if cut to 32 bits
    d = dict(_tensors(), x=big(rows, 128), y=big(rows, 64), index=None, out=None, h=None)
    with pytest.raises(ValueError, match="beyond 32 bits"):
        w4.w4a16_lora_forward(**d)
    with pytest.raises(ValueError, match="beyond 32 bits"):
        w4.w4a16_lora_forward(**dict(_tensors(), a=big(2 ** 32 + 2, 16, 128), b=big(2 ** 32 + 2, 64, 16)))
    with pytest.raises(ValueError, match="beyond 32 bits"):
        w4.w4a16_act_quantize(big(rows, 128), 32)
    with pytest.raises(ValueError, match="beyond 32 bits"):
        w4.w4a16_act_dequantize(big(rows, 128, dtype=torch.uint8), big(rows, 4), 32)
    b = _backward_tensors()
    with pytest.raises(ValueError, match="beyond 32 bits"):
        w4.w4a16_lora_backward(**dict(b, dy=big(rows, 64), x=big(rows, 128), h=big(rows, 16, dtype=torch.float32)))


def test_missing_operands_are_refused():
    for name in ("y", "x", "a", "b"):
        with pytest.raises((TypeError, ValueError)):
            w4.w4a16_lora_forward(**dict(_tensors(), **{name: None}))
    for name in ("dy", "x", "a", "b", "h"):
        with pytest.raises((TypeError, ValueError)):
            w4.w4a16_lora_backward(**dict(_backward_tensors(), **{name: None}))


# Sizes within the bounds of every argument whose grids would pass 2^32 threads, or the int that
# holds their workgroups: the output stream of the forward and of the input's gradient, and the
# gradients of many adapters.  Too small a workspace keeps them off the device in any case.
LARGE_FORWARD = [dict(M=1 << 27, N=1 << 24, K=8), dict(M=1 << 27, N=(1 << 24) - 8, K=64), dict(M=1 << 26, N=1 << 23, K=8, L=65535)]
LARGE_BACKWARD = [dict(M=1 << 27, N=8, K=1 << 24), dict(M=1 << 27, N=64, K=(1 << 24) - 8), dict(M=64, N=1 << 20, K=8, L=65535)]


@pytest.mark.parametrize("sizes", LARGE_FORWARD)
def test_forward_refuses_grids_beyond_the_launch_limits(sizes):
    lib = adapters._lib()
    c = dict(FORWARD, **sizes, bytes=0, workspace=None)
    assert lib.w4a16_lora_forward(*c.values()) == w4.ERR_UNSUPPORTED
    assert lib.w4a16_lora_forward_workspace(c["M"], c["N"], c["K"], c["R"], c["L"], 1) == 0


@pytest.mark.parametrize("sizes", LARGE_BACKWARD)
def test_backward_refuses_grids_beyond_the_launch_limits(sizes):
    lib = adapters._lib()
    c = dict(BACKWARD, **sizes, bytes=0, workspace=None)
    assert lib.w4a16_lora_backward(*c.values()) == w4.ERR_UNSUPPORTED
    assert lib.w4a16_lora_backward_workspace(c["M"], c["N"], c["K"], c["R"], c["L"], 1) == 0


def test_largest_grids_that_a_device_can_hold_are_taken():
    """Operands of about 256 GB each, more than one GPU holds together.  (The gradients of many
    adapters are bounded by L (N + K) < 2^30 besides.)"""
    lib = adapters._lib()
    for M, N, K, L in ((1 << 27, 1024, 8, 1), (8192, 1 << 24, 8, 1), (512, 1 << 18, 8, 65535), (1 << 27, 8, 1024, 65535)):
        assert lib.w4a16_lora_forward_workspace(M, N, K, 8, L, 1) > 0, (M, N, K, L)
    for M, N, K, L in ((1 << 27, 8, 1024, 1), (8192, 8, 1 << 24, 1), (512, 8, 1 << 13, 65535), (1 << 27, 1024, 8, 65535)):
        assert lib.w4a16_lora_backward_workspace(M, N, K, 8, L, 1) > 0, (M, N, K, L)
