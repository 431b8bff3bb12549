"""Binding of the softmax cross entropy over a quantised vocabulary head
(include/w4a16_head.h, part of libw4a16.so): argument checks and marshalling, as for the
mixtures of experts."""

from __future__ import annotations

import ctypes
import functools

from .adapters import _check, _handle, _int32, _matrix, _on, _operands, _overlap, _ptr, _torch, _workspace
from .experts import _inputs, _layer_specs

_p, _i, _z = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t

_LOSS = (_i, [_p] * 5 + [_i, _p] + [_i] * 4 + [_p, _p, _p, _z, _p])
_LOSS_BACKWARD = (_i, [_p] * 6 + [_i, _p, _p] + [_i] * 4 + [_p, _p, _z, _p])

SIGNATURES = {
    "w4a16_head_loss_workspace": (_z, [_i] * 4),
    "w4a16_head_loss": _LOSS,
    "w8a16_head_loss": _LOSS,
    "w4a16_head_loss_backward_workspace": (_z, [_i] * 4),
    "w4a16_head_loss_backward": _LOSS_BACKWARD,
    "w8a16_head_loss_backward": _LOSS_BACKWARD,
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


@functools.lru_cache(maxsize=4096)
def _workspace_bytes(name, *sizes):
    return getattr(_lib(), name)(*sizes)


def _loss(bits, x, qweight, scales, qzeros, g_idx, group_size, target, vocab, loss, lse, stream):
    torch = _torch()
    M, K = _matrix(x, "x")
    _, N, layer = _layer_specs(qweight, scales, qzeros, g_idx, group_size, K, bits, False)
    vocab = N if vocab is None else _int32(vocab, "vocab")
    f32 = torch.float32
    specs = ((x, torch.float16, (M, K), "x"), *layer, (target, torch.int32, (M,), "target"))
    if target is None:
        raise TypeError("target must be a torch.int32 tensor")
    device = _operands((*specs, (loss, f32, (M,), "loss"), (lse, f32, (M,), "lse")))
    if loss is not None:
        _overlap(loss, *_inputs(specs), (lse, "lse"))
    if lse is not None:
        _overlap(lse, *_inputs(specs))
    with _on(device, stream):
        if loss is None:
            loss = torch.empty(M, dtype=f32, device=device)
        if lse is None:
            lse = torch.empty(M, dtype=f32, device=device)
        need = _workspace_bytes("w4a16_head_loss_workspace", M, N, K, int(g_idx is not None))
        ws = _workspace(max(need, 1), device)
        _check(getattr(_lib(), f"w{bits}a16_head_loss")(
            x.data_ptr(), qweight.data_ptr(), scales.data_ptr(), _ptr(qzeros), _ptr(g_idx), group_size,
            target.data_ptr(), M, N, K, vocab, loss.data_ptr(), lse.data_ptr(), ws.data_ptr(), need, _handle(device)))
    return loss, lse


def w4a16_head_loss(x, qweight, scales, qzeros, g_idx, group_size: int, target, vocab=None, loss=None, lse=None,
                    stream=None):
    """Softmax cross entropy of the rows of x binary16 [M][K] under a packed head of N rows, of
    which the first vocab (None: all) are classes: (loss float32 [M], lse float32 [M]), lse the
    logarithm of the sum of exponentials that the backward pass takes.  target int32 [M]; a
    value outside [0, vocab) (-100 by convention) is a row without a target: loss and lse 0.
    The logits are never written."""
    return _loss(4, x, qweight, scales, qzeros, g_idx, group_size, target, vocab, loss, lse, stream)


def w8a16_head_loss(x, qweight, scales, qzeros, g_idx, group_size: int, target, vocab=None, loss=None, lse=None,
                    stream=None):
    """w4a16_head_loss for an 8-bit head."""
    return _loss(8, x, qweight, scales, qzeros, g_idx, group_size, target, vocab, loss, lse, stream)


def _loss_backward(bits, dloss, x, qweight, scales, qzeros, g_idx, group_size, target, lse, vocab, out, stream):
    torch = _torch()
    M, K = _matrix(x, "x")
    _, N, layer = _layer_specs(qweight, scales, qzeros, g_idx, group_size, K, bits, False)
    vocab = N if vocab is None else _int32(vocab, "vocab")
    f32 = torch.float32
    specs = ((x, torch.float16, (M, K), "x"), *layer, (target, torch.int32, (M,), "target"), (lse, f32, (M,), "lse"),
             (dloss, f32, (M,), "dloss"))
    if target is None or lse is None or dloss is None:
        raise TypeError("target must be a torch.int32 tensor, lse and dloss torch.float32 tensors")
    device = _operands((*specs, (out, torch.float16, (M, K), "out")))
    if out is not None:
        _overlap(out, *_inputs(specs))
    with _on(device, stream):
        if out is None:
            out = torch.empty((M, K), dtype=torch.float16, device=device)
        need = _workspace_bytes("w4a16_head_loss_backward_workspace", M, N, K, int(g_idx is not None))
        ws = _workspace(max(need, 1), device)
        _check(getattr(_lib(), f"w{bits}a16_head_loss_backward")(
            dloss.data_ptr(), x.data_ptr(), qweight.data_ptr(), scales.data_ptr(), _ptr(qzeros), _ptr(g_idx),
            group_size, target.data_ptr(), lse.data_ptr(), M, N, K, vocab, out.data_ptr(), ws.data_ptr(), need,
            _handle(device)))
    return out


def w4a16_head_loss_backward(dloss, x, qweight, scales, qzeros, g_idx, group_size: int, target, lse, vocab=None,
                             out=None, stream=None):
    """Gradient of x for dloss float32 [M], that of the losses (with the training program's loss
    scale in it): binary16 [M][K].  The other arguments as in w4a16_head_loss, lse what it
    returned.  Logits are computed again, piece by piece of the vocabulary."""
    return _loss_backward(4, dloss, x, qweight, scales, qzeros, g_idx, group_size, target, lse, vocab, out, stream)


def w8a16_head_loss_backward(dloss, x, qweight, scales, qzeros, g_idx, group_size: int, target, lse, vocab=None,
                             out=None, stream=None):
    """w4a16_head_loss_backward for an 8-bit head."""
    return _loss_backward(8, dloss, x, qweight, scales, qzeros, g_idx, group_size, target, lse, vocab, out, stream)
