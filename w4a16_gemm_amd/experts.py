"""Binding of the mixtures of experts (include/w4a16_experts.h, part of libw4a16.so):
argument checks and marshalling, as for the adapters.  Device tensors only; the workspace
of a call comes from torch's allocator on the call's stream, so a call can be captured into
a graph (which then holds its own workspace) and calls on different streams share nothing."""

from __future__ import annotations

import ctypes
import functools

from .adapters import (_check, _handle, _int32, _matrix, _on, _operands, _overlap, _ptr, _sizes, _torch, _workspace)

_p, _i, _z = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t

_FORWARD = (_i, [_p] * 5 + [_i, _p] + [_i] * 5 + [_p, _p, _z, _p])
_BACKWARD = (_i, [_p] * 5 + [_i, _p, _p] + [_i] * 5 + [_p, _p, _z, _p])
_LAYER_BACKWARD = (_i, [_p] * 5 + [_i, _p] + [_i] * 3 + [_p, _p, _z, _p])

SIGNATURES = {
    "w4a16_route": (_i, [_p] + [_i] * 5 + [_p] * 3),
    "w4a16_route_backward": (_i, [_p, _p, _i, _p, _p] + [_i] * 4 + [_p, _p]),
    "w4a16_experts_gemm_workspace": (_z, [_i] * 6),
    "w4a16_experts_gemm": _FORWARD,
    "w8a16_experts_gemm": _FORWARD,
    "w4a16_experts_backward_workspace": (_z, [_i] * 6),
    "w4a16_experts_backward": _BACKWARD,
    "w8a16_experts_backward": _BACKWARD,
    "w4a16_gemm_backward": _LAYER_BACKWARD,
    "w8a16_gemm_backward": _LAYER_BACKWARD,
    "w4a16_experts_combine": (_i, [_p, _p, _i, _i, _i, _p, _p]),
    "w4a16_experts_combine_backward": (_i, [_p, _p, _p, _i, _i, _i, _p, _p, _p]),
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


@functools.lru_cache(maxsize=4096)
def _words(bits, N, K, act):
    from . import lib
    return getattr(lib(), f"w{bits}a16_qweight_words")(N, K, act)


def _layer_specs(qweight, scales, qzeros, g_idx, group_size, K, bits, experts):
    """(E, N, specs) of the packed weights: one layer (experts False: no leading size, E = 1)
    or a stack of them.  Sizes that the library refuses are left to it."""
    torch = _torch()
    sizes = _sizes(scales, 3 if experts else 2, "scales [E][G][N]" if experts else "scales [G][N]")
    E, N = sizes[0] if experts else 1, sizes[-1]
    if group_size <= 0 or K <= 0 or K % group_size:
        raise ValueError(f"K={K} is not a positive multiple of group_size={group_size}")
    G = K // group_size
    words = _words(bits, N, K, int(g_idx is not None))
    if words == 0:
        raise ValueError(f"no packed layer has N={N} outputs and K={K} channels")
    if qweight is None or scales is None:
        raise TypeError("qweight must be a torch.int32 tensor and scales a torch.float16 tensor")
    lead = (E,) if experts else ()
    if not experts and isinstance(qweight, torch.Tensor) and qweight.dtype == torch.int32 and qweight.numel() >= words:
        words = qweight.numel()     # as the layer's own calls: at least the words of the layer
        lead = ()
    return E, N, ((qweight, torch.int32, lead + (words,), "qweight"), (scales, torch.float16, lead + (G, N), "scales"),
                  (qzeros, torch.int32, lead + (G, N * bits // 32), "qzeros"),
                  (g_idx, torch.int32, lead + (K,), "g_idx"))


def _inputs(specs):
    return tuple((s[0], s[3]) for s in specs)


def _slots(index):
    """(M, T, leading shape) of index [M][T] or [M]."""
    if not isinstance(index, _torch().Tensor) or index.dim() not in (1, 2):
        raise ValueError("index must be a [M][T] or [M] tensor")
    shape = tuple(index.shape)
    if max(shape) > 2 ** 31 - 1:
        raise ValueError(f"index has shape {shape}, a size beyond 32 bits")
    return (shape[0], 1, shape) if index.dim() == 1 else (shape[0], shape[1], shape)


def _logit_bits(logits):
    torch = _torch()
    if not isinstance(logits, torch.Tensor) or logits.dtype not in (torch.float16, torch.float32):
        raise TypeError("logits must be a torch.float16 or torch.float32 tensor")
    return 16 if logits.dtype == torch.float16 else 32


def w4a16_route(logits, top_k: int, renormalise: bool = True, index=None, weights=None, stream=None):
    """Experts of every row: (index int32 [M][top_k], weights float32 [M][top_k]) from logits
    [M][E], binary16 or float32: the top_k largest of softmax(logits) in descending order, of
    equal ones the lower index first; renormalise divides a row's weights by their sum.
    Experts with the logit -infinity are never chosen; rows left short get -1 and 0."""
    torch = _torch()
    bits = _logit_bits(logits)
    M, E = _matrix(logits, "logits")
    top_k = _int32(top_k, "top_k")
    device = _operands(((logits, logits.dtype, (M, E), "logits"), (index, torch.int32, (M, top_k), "index"),
                        (weights, torch.float32, (M, top_k), "weights")))
    if index is not None:
        _overlap(index, (logits, "logits"), (weights, "weights"))
    if weights is not None:
        _overlap(weights, (logits, "logits"))
    with _on(device, stream):
        if index is None:
            index = torch.empty((M, max(top_k, 0)), dtype=torch.int32, device=device)
        if weights is None:
            weights = torch.empty((M, max(top_k, 0)), dtype=torch.float32, device=device)
        _check(_lib().w4a16_route(logits.data_ptr(), bits, M, E, top_k, int(bool(renormalise)), index.data_ptr(),
                                  weights.data_ptr(), _handle(device)))
    return index, weights


def w4a16_route_backward(dweights, logits, index, weights, renormalise: bool = True, out=None, stream=None):
    """Gradient of the logits (their type and shape) for dweights float32 [M][top_k]; index and
    weights as w4a16_route gave them."""
    torch = _torch()
    bits = _logit_bits(logits)
    M, E = _matrix(logits, "logits")
    top_k = _matrix(index, "index")[1]
    f32 = torch.float32
    device = _operands(((logits, logits.dtype, (M, E), "logits"), (index, torch.int32, (M, top_k), "index"),
                        (weights, f32, (M, top_k), "weights"), (dweights, f32, (M, top_k), "dweights"),
                        (out, logits.dtype, (M, E), "out")))
    if dweights is None or weights is None:
        raise TypeError("dweights and weights must be torch.float32 tensors")
    if out is not None:
        _overlap(out, (logits, "logits"), (index, "index"), (weights, "weights"), (dweights, "dweights"))
    with _on(device, stream):
        if out is None:
            out = torch.empty_like(logits)
        _check(_lib().w4a16_route_backward(dweights.data_ptr(), logits.data_ptr(), bits, index.data_ptr(),
                                           weights.data_ptr(), M, E, top_k, int(bool(renormalise)), out.data_ptr(),
                                           _handle(device)))
    return out


def _gemm(bits, x, qweight, scales, qzeros, g_idx, group_size, index, out, stream):
    torch = _torch()
    M, K = _matrix(x, "x")
    rows, T, lead = _slots(index)
    E, N, layer = _layer_specs(qweight, scales, qzeros, g_idx, group_size, K, bits, True)
    specs = ((x, torch.float16, (rows, K), "x"), *layer, (index, torch.int32, lead, "index"))
    device = _operands((*specs, (out, torch.float16, lead + (N,), "out")))
    if out is not None:
        _overlap(out, *_inputs(specs))
    with _on(device, stream):
        if out is None:
            out = torch.empty(lead + (N,), dtype=torch.float16, device=device)
        need = _workspace_bytes("w4a16_experts_gemm_workspace", M, T, E, N, K, int(g_idx is not None))
        ws = _workspace(need, device)
        _check(getattr(_lib(), f"w{bits}a16_experts_gemm")(
            x.data_ptr(), qweight.data_ptr(), scales.data_ptr(), _ptr(qzeros), _ptr(g_idx), group_size,
            index.data_ptr(), M, T, E, N, K, out.data_ptr(), _ptr(ws), need, _handle(device)))
    return out


def w4a16_experts_gemm(x, qweight, scales, qzeros, g_idx, group_size: int, index, out=None, stream=None):
    """y[m][t] = W^_e x[m] with e = index[m][t]: binary16 [M][T][N] ([M][N] for index [M]).

    x binary16 [M][K]; the experts' packed layers one after the other: qweight int32 [E][words]
    (w4a16_pack of every expert), scales binary16 [E][G][N], qzeros int32 [E][G][N/8] or None
    (symmetric), g_idx int32 [E][K] or None (act order, every expert its own); index int32, a
    value outside [0, E) (-1 by convention) is a slot without an expert and gets zeros."""
    return _gemm(4, x, qweight, scales, qzeros, g_idx, group_size, index, out, stream)


def w8a16_experts_gemm(x, qweight, scales, qzeros, g_idx, group_size: int, index, out=None, stream=None):
    """w4a16_experts_gemm for 8-bit weights (qzeros int32 [E][G][N/4] or None)."""
    return _gemm(8, x, qweight, scales, qzeros, g_idx, group_size, index, out, stream)


def _backward(bits, dy, qweight, scales, qzeros, g_idx, group_size, index, K, dx, out, stream):
    torch = _torch()
    f16 = torch.float16
    experts = index is not None
    E, N, layer = _layer_specs(qweight, scales, qzeros, g_idx, group_size, K, bits, experts)
    if experts:
        M, T, lead = _slots(index)
    else:
        M, T = _matrix(dy, "dy")[0], 1
        lead = (M,)
    specs = ((dy, f16, lead + (N,), "dy"), *layer, (index, torch.int32, lead, "index"))
    device = _operands((*specs, (dx, f16, (M, K), "dx"), (out, f16, (M, K), "out")))
    if dy is None:
        raise TypeError("dy must be a torch.float16 tensor")
    if out is not None:
        if dx is not None and out.data_ptr() != dx.data_ptr():
            _overlap(out, (dx, "dx"))
        _overlap(out, *_inputs(specs))
    with _on(device, stream):
        if out is None:
            out = torch.empty((M, K), dtype=f16, device=device)
        need = _workspace_bytes("w4a16_experts_backward_workspace", M, T, E, N, K, int(g_idx is not None))
        ws = _workspace(max(need, 1), device)
        weights = (dy.data_ptr(), qweight.data_ptr(), scales.data_ptr(), _ptr(qzeros), _ptr(g_idx), group_size)
        tail = (out.data_ptr(), ws.data_ptr(), need, _handle(device))
        if experts:
            _check(getattr(_lib(), f"w{bits}a16_experts_backward")(*weights, index.data_ptr(), _ptr(dx), M, T, E, N, K,
                                                                   *tail))
        else:
            _check(getattr(_lib(), f"w{bits}a16_gemm_backward")(*weights, _ptr(dx), M, N, K, *tail))
    return out


def w4a16_experts_backward(dy, qweight, scales, qzeros, g_idx, group_size: int, index, K: int, dx=None, out=None,
                           stream=None):
    """Gradient of w4a16_experts_gemm's rows for dy binary16 [M][T][N]: binary16 [M][K], the sum
    over a row's slots of W^_e^T dy[m][t].  dx binary16 [M][K] is a gradient that already
    reaches x and is added to (None: 0); the sum goes to out (allocated unless given; out=dx
    works in place).  Rows of dy without an expert are not read."""
    if index is None:
        raise ValueError("index must be a [M][T] or [M] tensor")
    return _backward(4, dy, qweight, scales, qzeros, g_idx, group_size, index, K, dx, out, stream)


def w8a16_experts_backward(dy, qweight, scales, qzeros, g_idx, group_size: int, index, K: int, dx=None, out=None,
                           stream=None):
    """w4a16_experts_backward for 8-bit weights."""
    if index is None:
        raise ValueError("index must be a [M][T] or [M] tensor")
    return _backward(8, dy, qweight, scales, qzeros, g_idx, group_size, index, K, dx, out, stream)


def w4a16_gemm_backward(dy, qweight, scales, qzeros, g_idx, group_size: int, K: int, dx=None, out=None, stream=None):
    """Gradient of w4a16_gemm's x through the frozen weights: binary16(dx + dy W^) [M][K] for dy
    binary16 [M][N], without W^ in memory.  dx and out as in w4a16_experts_backward."""
    return _backward(4, dy, qweight, scales, qzeros, g_idx, group_size, None, K, dx, out, stream)


def w8a16_gemm_backward(dy, qweight, scales, qzeros, g_idx, group_size: int, K: int, dx=None, out=None, stream=None):
    """w4a16_gemm_backward for 8-bit weights."""
    return _backward(8, dy, qweight, scales, qzeros, g_idx, group_size, None, K, dx, out, stream)


def w4a16_experts_combine(y, weights, out=None, stream=None):
    """out[m] = sum_t weights[m][t] y[m][t]: binary16 [M][N] from y binary16 [M][T][N] and weights
    float32 [M][T]."""
    torch = _torch()
    M, T, N = _sizes(y, 3, "y [M][T][N]")
    specs = ((y, torch.float16, (M, T, N), "y"), (weights, torch.float32, (M, T), "weights"))
    if weights is None:
        raise TypeError("weights must be a torch.float32 tensor")
    device = _operands((*specs, (out, torch.float16, (M, N), "out")))
    if out is not None:
        _overlap(out, *_inputs(specs))
    with _on(device, stream):
        if out is None:
            out = torch.empty((M, N), dtype=torch.float16, device=device)
        _check(_lib().w4a16_experts_combine(y.data_ptr(), weights.data_ptr(), M, T, N, out.data_ptr(), _handle(device)))
    return out


def w4a16_experts_combine_backward(dout, y, weights, stream=None):
    """Gradients of w4a16_experts_combine for dout binary16 [M][N]: (dy binary16 [M][T][N],
    dweights float32 [M][T])."""
    torch = _torch()
    M, T, N = _sizes(y, 3, "y [M][T][N]")
    if weights is None or dout is None:
        raise TypeError("dout must be a torch.float16 tensor and weights a torch.float32 tensor")
    device = _operands(((y, torch.float16, (M, T, N), "y"), (weights, torch.float32, (M, T), "weights"),
                        (dout, torch.float16, (M, N), "dout")))
    with _on(device, stream):
        dy = torch.empty_like(y)
        dweights = torch.empty_like(weights)
        _check(_lib().w4a16_experts_combine_backward(dout.data_ptr(), y.data_ptr(), weights.data_ptr(), M, T, N,
                                                     dy.data_ptr(), dweights.data_ptr(), _handle(device)))
    return dy, dweights
