"""Binding of the low-rank adapters and the 8-bit activation checkpoints
(include/w4a16_adapters.h, part of libw4a16.so): argument checks and marshalling, as for
the layer itself.  Device tensors only; the workspace of a call comes from torch's
allocator on the call's stream, so a call can be captured into a graph (which then holds
its own workspace) and calls on different streams share nothing."""

from __future__ import annotations

import contextlib
import ctypes
import functools

_p, _i, _z = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t

SIGNATURES = {
    "w4a16_lora_forward_workspace": (_z, [_i] * 6),
    "w4a16_lora_forward": (_i, [_p] * 6 + [_i] * 5 + [_p] * 3 + [_z, _p]),
    "w4a16_lora_backward_workspace": (_z, [_i] * 6),
    "w4a16_lora_backward": (_i, [_p] * 8 + [_i] * 5 + [_p] * 4 + [_z, _p]),
    "w4a16_lora_backward_q8": (_i, [_p] * 3 + [_i] + [_p] * 6 + [_i] * 5 + [_p] * 4 + [_z, _p]),
    "w4a16_act_quantize": (_i, [_p, _i, _i, _i, _p, _p, _p]),
    "w4a16_act_dequantize": (_i, [_p, _p, _i, _i, _i, _p, _p]),
}


@functools.lru_cache(maxsize=None)
def _lib():
    from . import lib
    handle = lib()
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(handle, name)
        fn.restype = res
        fn.argtypes = args
    return handle


def _check(status: int) -> None:
    if status:
        from . import W4A16Error
        raise W4A16Error(status, _lib().w4a16_last_error().decode())


def _operands(specs):
    """Check (tensor, dtype, shape, name) rows, skipping absent tensors: types and shapes
    first, then that all of them are contiguous and on one ROCm device.  Returns it."""
    Tensor = _torch().Tensor
    for t, dtype, shape, name in specs:
        if t is not None:
            if not isinstance(t, Tensor) or t.dtype != dtype:
                raise TypeError(f"{name} must be a {dtype} tensor")
            if t.shape != shape:
                raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {shape}")
    device = None
    for t, dtype, shape, name in specs:
        if t is not None:
            if not t.is_contiguous():
                raise TypeError(f"{name} must be contiguous")
            if device is None:
                if not t.is_cuda:
                    raise TypeError(f"{name} must live on a ROCm device")
                device = t.device
            elif t.device != device:
                if not t.is_cuda:
                    raise TypeError(f"{name} must live on a ROCm device")
                raise ValueError(f"{name} is on {t.device}, the other tensors on {device}")
    return device


@functools.lru_cache(maxsize=None)
def _torch():
    import torch
    return torch


@contextlib.contextmanager
def _other(device, stream):
    torch = _torch()
    with torch.cuda.device(device), torch.cuda.stream(stream):
        yield


_HERE = contextlib.nullcontext()


def _on(device, stream):
    """Context in which `device` is current and allocations belong to the call's stream."""
    cuda = _torch().cuda
    if stream is not None:
        if stream.device != device:
            raise ValueError(f"stream of {stream.device}, tensors on {device}")
        return _other(device, stream)
    if cuda.current_device() != device.index:
        return cuda.device(device)
    return _HERE


def _handle(device):
    """Raw handle of the device's current stream (torch's own accessor for it where there is
    one: the Stream object costs 1.7 us more)."""
    raw = getattr(_torch()._C, "_cuda_getCurrentRawStream", None)
    return _torch().cuda.current_stream(device).cuda_stream if raw is None else raw(device.index)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _sizes(t, dims, name):
    """The shape, whose entries have to fit the int arguments of the library."""
    if not isinstance(t, _torch().Tensor) or t.dim() != dims:
        raise ValueError(f"{name} must be a {dims}-d tensor")
    if max(t.shape) > 2 ** 31 - 1:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, a size beyond 32 bits")
    return t.shape


def _matrix(t, name):
    return _sizes(t, 2, name)


def _adapter_sizes(a, b):
    L, R = _sizes(a, 3, "a [L][R][K]")[:2]
    _sizes(b, 3, "b [L][N][R]")
    return L, R


def _overlap(out, *others):
    """Refuse an output that shares memory with another operand."""
    lo, hi = out.data_ptr(), out.data_ptr() + out.numel() * out.element_size()
    for t, name in others:
        if t is not None and t.data_ptr() < hi and lo < t.data_ptr() + t.numel() * t.element_size():
            raise ValueError(f"an output overlaps {name}")


@functools.lru_cache(maxsize=4096)
def _workspace_bytes(name, *sizes):
    return getattr(_lib(), name)(*sizes)


def _workspace(nbytes, device):
    torch = _torch()
    return torch.empty(nbytes, dtype=torch.uint8, device=device) if nbytes else None


def w4a16_lora_forward(y, x, a, b, index=None, scaling=None, out=None, h=None, stream=None):
    """out[m] = binary16(y[m] + s_i B_i (A_i x[m])) with i = index[m].

    y binary16 [M][N] is the shared projection's output (w4a16_gemm or w8a16_gemm of the
    same x), x binary16 [M][K], a binary16 [L][R][K], b binary16 [L][N][R]; R a multiple of
    8 up to 128.  index int32 [M] (None: adapter 0 everywhere; -1 or any value outside [0,
    L): no adapter, the row passes through); scaling float32 [L] (None: 1).  Returns out
    (allocated unless given; out=y works in place).  h float32 [M][R], if given, receives
    A_i x for the backward pass."""
    torch = _torch()
    M, K = _matrix(x, "x")
    N = _matrix(y, "y")[1]
    L, R = _adapter_sizes(a, b)
    f16, f32 = torch.float16, torch.float32
    device = _operands(((x, f16, (M, K), "x"), (y, f16, (M, N), "y"), (a, f16, (L, R, K), "a"), (b, f16, (L, N, R), "b"),
                        (index, torch.int32, (M,), "index"), (scaling, f32, (L,), "scaling"),
                        (out, f16, (M, N), "out"), (h, f32, (M, R), "h")))
    if out is not None or h is not None:
        ins = ((x, "x"), (a, "a"), (b, "b"), (index, "index"), (scaling, "scaling"))
        if out is not None:
            if out.data_ptr() != y.data_ptr():
                _overlap(out, (y, "y"))
            _overlap(out, *ins, (h, "h"))
        if h is not None:
            _overlap(h, *ins, (y, "y"))
    with _on(device, stream):
        if out is None:
            out = torch.empty_like(y)
        need = _workspace_bytes("w4a16_lora_forward_workspace", M, N, K, R, L, index is not None)
        ws = _workspace(need, device)
        _check(_lib().w4a16_lora_forward(y.data_ptr(), x.data_ptr(), a.data_ptr(), b.data_ptr(), _ptr(index),
                                         _ptr(scaling), M, N, K, R, L, out.data_ptr(), _ptr(h), _ptr(ws), need,
                                         _handle(device)))
    return out


def _backward(dy, kept, specs, K, a, b, h, index, scaling, dx, out, need_dx, stream, entry):
    torch = _torch()
    M, N = _matrix(dy, "dy")
    L, R = _adapter_sizes(a, b)
    f16, f32 = torch.float16, torch.float32
    if h is None:
        raise TypeError("h must be a torch.float32 tensor")
    device = _operands(((dy, f16, (M, N), "dy"), *specs, (a, f16, (L, R, K), "a"), (b, f16, (L, N, R), "b"),
                        (h, f32, (M, R), "h"), (index, torch.int32, (M,), "index"), (scaling, f32, (L,), "scaling"),
                        (dx, f16, (M, K), "dx"), (out, f16, (M, K), "out")))
    if not need_dx and (dx is not None or out is not None):
        raise ValueError("need_dx=False takes neither dx nor out")
    if out is not None:
        if dx is not None and out.data_ptr() != dx.data_ptr():
            _overlap(out, (dx, "dx"))
        _overlap(out, (dy, "dy"), (a, "a"), (b, "b"), (h, "h"), (index, "index"), (scaling, "scaling"),
                 *((s[0], s[3]) for s in specs))
    with _on(device, stream):
        if need_dx and out is None:
            out = torch.empty((M, K), dtype=f16, device=device)
        da = torch.empty((L, R, K), dtype=f32, device=device)
        db = torch.empty((L, N, R), dtype=f32, device=device)
        need = _workspace_bytes("w4a16_lora_backward_workspace", M, N, K, R, L, index is not None)
        ws = _workspace(need, device)
        _check(getattr(_lib(), entry)(dy.data_ptr(), *kept, a.data_ptr(), b.data_ptr(), h.data_ptr(), _ptr(index),
                                      _ptr(scaling), _ptr(dx), M, N, K, R, L, _ptr(out), da.data_ptr(), db.data_ptr(),
                                      _ptr(ws), need, _handle(device)))
    return out, da, db


def w4a16_lora_backward(dy, x, a, b, h, index=None, scaling=None, dx=None, out=None, need_dx=True, stream=None):
    """Gradients of w4a16_lora_forward for dy binary16 [M][N]: (dx binary16 [M][K], da
    float32 [L][R][K], db float32 [L][N][R]).  x, a, b, index and scaling as in the
    forward call, h what it wrote.  dx binary16 [M][K] is the gradient that already reaches
    x (through the quantised weights) and is added to (None: 0); the sum goes to out
    (allocated unless given; out=dx works in place).  need_dx=False: dx is not computed and
    None is returned in its place."""
    M, K = _matrix(x, "x")
    return _backward(dy, (x.data_ptr(),), ((x, _torch().float16, (_matrix(dy, "dy")[0], K), "x"),), K, a, b, h, index,
                     scaling, dx, out, need_dx, stream, "w4a16_lora_backward")


def w4a16_lora_backward_q8(dy, codes, scales, group_size: int, a, b, h, index=None, scaling=None, dx=None, out=None,
                           need_dx=True, stream=None):
    """w4a16_lora_backward with x as an 8-bit checkpoint (codes, scales of
    w4a16_act_quantize): the same bits as from the restored x, which is never stored."""
    K = _matrix(codes, "codes")[1]
    rows = _matrix(dy, "dy")[0]
    specs = _checkpoint(codes, scales, group_size, rows, K)
    return _backward(dy, (codes.data_ptr(), scales.data_ptr(), group_size), specs, K, a, b, h, index, scaling, dx, out,
                     need_dx, stream, "w4a16_lora_backward_q8")


def _checkpoint(codes, scales, group_size, M, K):
    """Specs of a checkpoint's tensors (groups of a size that does not divide K are left to
    the library to refuse)."""
    torch = _torch()
    G = K // group_size if group_size > 0 else 0
    if scales is None:
        raise TypeError("scales must be a torch.float16 tensor")
    return (codes, torch.uint8, (M, K), "codes"), (scales, torch.float16, (M, G), "scales")


def w4a16_act_quantize(x, group_size: int, codes=None, scales=None, stream=None):
    """Keep x binary16 [M][K] in 8 bits: (codes uint8 [M][K], scales binary16
    [M][K/group_size]), group_size 32, 64 or 128 (allocated unless given)."""
    torch = _torch()
    M, K = _matrix(x, "x")
    G = K // group_size if group_size > 0 else 0
    device = _operands(((x, torch.float16, (M, K), "x"), (codes, torch.uint8, (M, K), "codes"),
                        (scales, torch.float16, (M, G), "scales")))
    if codes is not None:
        _overlap(codes, (x, "x"), (scales, "scales"))
    if scales is not None:
        _overlap(scales, (x, "x"))
    with _on(device, stream):
        if codes is None:
            codes = torch.empty((M, K), dtype=torch.uint8, device=device)
        if scales is None:
            scales = torch.empty((M, G), dtype=torch.float16, device=device)
        _check(_lib().w4a16_act_quantize(x.data_ptr(), M, K, group_size, codes.data_ptr(), scales.data_ptr(),
                                         _handle(device)))
    return codes, scales


def w4a16_act_dequantize(codes, scales, group_size: int, out=None, stream=None):
    """binary16 [M][K] from a checkpoint: binary16((codes - 128) * scale)."""
    torch = _torch()
    M, K = _matrix(codes, "codes")
    specs = _checkpoint(codes, scales, group_size, M, K)
    device = _operands((*specs, (out, torch.float16, (M, K), "out")))
    if out is not None:
        _overlap(out, (codes, "codes"), (scales, "scales"))
    with _on(device, stream):
        if out is None:
            out = torch.empty((M, K), dtype=torch.float16, device=device)
        _check(_lib().w4a16_act_dequantize(codes.data_ptr(), scales.data_ptr(), M, K, group_size, out.data_ptr(),
                                           _handle(device)))
    return out
