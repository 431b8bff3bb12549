"""Cases of the adapter operators beside the quantised linear layer: low-rank adapters of
many requests, their backward pass, and activation checkpoints in 8 bits.

``run`` makes one pass.  With ``own`` false it computes the operators in elementary torch
operations in 32 bits; with ``own`` true it calls the library.  ``exact`` computes the same
outputs in 64 bits from the definitions:

  forward     out[m] = binary16(y[m] + s_i B_i (A_i x[m])), i = index[m]; rows without an
              adapter (i = -1) pass through; h[m] = A_i x[m]
  backward    g[m] = B_i^T dy[m];  dx[m] = binary16(dx0[m] + s_i A_i^T g[m]);
              dB_i = s_i sum dy[m] h[m]^T;  dA_i = s_i sum g[m] x[m]^T
  checkpoint  per row and group of g channels: S = smallest binary16 >= max|x| / 127
              (1 for a group of zeros), q = round(x / S) half to even, value binary16(q S)
"""

import math

import torch

own = False


def listed():
    """Layer shapes: 1536 -> 1536 and 1536 -> 8960 (o and up projections of the 1.5B-class
    model), 4096 -> 11008, 4096 -> 14336 and 8192 -> 28672 (the layer configurations)."""
    return [
        # decode, one sequence, a small projection: only latency counts
        dict(name="forward_one_row", op="forward", M=1, K=1536, N=1536, R=16, L=4, order="mixed", bare=0.0),
        # decode of 16 sequences on the largest projection, every row of 8 adapters
        dict(name="forward_decode", op="forward", M=16, K=8192, N=28672, R=16, L=8, order="mixed", bare=0.0),
        # a ragged serving batch: rows in no order, a fifth of them without an adapter
        dict(name="forward_ragged", op="forward", M=77, K=4096, N=11008, R=24, L=12, order="mixed", bare=0.2),
        # prefill of eight requests, each with an adapter of its own
        dict(name="forward_prefill", op="forward", M=2048, K=4096, N=14336, R=64, L=8, order="runs", bare=0.0),
        # the input of a small layer kept in 8 bits and restored, finest groups, odd rows
        dict(name="checkpoint_small", op="checkpoint", M=33, K=1536, group=32),
        # the input of a large layer for a long batch
        dict(name="checkpoint_large", op="checkpoint", M=8192, K=8192, group=128),
        # fine-tuning one adapter, input kept in 16 bits
        dict(name="backward_half", op="backward", M=512, K=4096, N=11008, R=16, L=1, order="one", bare=0.0, group=0),
        # fine-tuning one adapter, input kept in 8 bits
        dict(name="backward_8bit", op="backward", M=2048, K=4096, N=14336, R=16, L=1, order="one", bare=0.0, group=128),
        # several adapters trained in one batch of ragged runs, some rows without one
        dict(name="backward_many", op="backward", M=1111, K=1536, N=8960, R=32, L=6, order="runs", bare=0.1, group=64),
        # a short batch on the wide-to-narrow projection, large rank
        dict(name="backward_rank128", op="backward", M=300, K=8960, N=1536, R=128, L=2, order="runs", bare=0.0, group=0),
        # one training step of an adapter on the largest layer: forward, checkpoint, backward
        dict(name="train_step", op="train", M=4096, K=8192, N=28672, R=64, L=1, order="one", bare=0.0, group=128),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["forward", "forward", "checkpoint", "backward", "backward", "train"])
    group = rng.choice([32, 64, 128])
    K = group * max(4, _log_int(rng, 512, 8960) // group)
    if op == "checkpoint":
        return dict(op=op, M=_log_int(rng, 1, 8192), K=K, group=group)
    M = _log_int(rng, 1 if op == "forward" else 64, 4096)
    N = 8 * _log_int(rng, 64, 3584)
    R = 8 * rng.randint(1, 16)
    order = rng.choice(["one", "mixed", "runs"])
    L = 1 if order == "one" else rng.randint(2, 16)
    bare = 0.0 if order == "one" else rng.choice([0.0, 0.1, 0.3])
    if op == "backward":
        group = rng.choice([0, group])
    case = dict(op=op, M=M, K=K, N=N, R=R, L=L, order=order, bare=bare)
    if op != "forward":
        case["group"] = group
    most = work(listed()[-1])
    while any(work(case)[k] > most[k] for k in most):
        case["M"] = max(1, case["M"] // 2)
    return case


# --- work of one pass -------------------------------------------------------------

def _adapted_rows(case):
    return case["M"] - int(case["M"] * case["bare"])


def work(case):
    M, K = case["M"], case["K"]
    if case["op"] == "checkpoint":
        # values in, codes and scales written and read, values out
        codes = M * K + 2 * M * (K // case["group"])
        return {"bytes": 4 * M * K + 2 * codes, "flops": 4 * M * K}
    N, R = case["N"], case["R"]
    rows = _adapted_rows(case)
    used = min(case["L"], rows)
    adapters = 2 * used * R * (K + N)
    kept = 0 if case["op"] == "forward" else 2 * M * K if not case["group"] else M * K + 2 * M * (K // case["group"])
    forward = {"bytes": 2 * rows * K + 4 * M * N + adapters, "flops": 2 * rows * R * (K + N)}
    backward = {"bytes": 2 * rows * N + kept + adapters + 4 * M * R + 4 * M * K + 4 * case["L"] * R * (K + N),
                "flops": 4 * rows * R * (K + N)}
    if case["op"] == "forward":
        return forward
    if case["op"] == "backward":
        return backward
    # a step: x, y, dy, dx0 and the adapters in; out, dx and the gradients out; the
    # checkpoint is written and read
    return {"bytes": 2 * M * K + 4 * M * N + 2 * M * N + 4 * M * K + 2 * kept + adapters + 4 * case["L"] * R * (K + N),
            "flops": forward["flops"] + backward["flops"] + 2 * M * K}


# --- inputs -----------------------------------------------------------------------

def _index(case, gen):
    """Adapter of every row: int32 [M] (None when there is one adapter for all rows)."""
    M, L = case["M"], case["L"]
    if case["order"] == "one":
        return None
    rows = _adapted_rows(case)
    index = torch.arange(rows) % L
    if case["order"] == "runs":
        # ragged runs: every adapter once, the rest of the rows dealt by random weights
        weight = torch.rand(L, generator=gen) + 0.2
        extra = (weight / weight.sum() * max(rows - L, 0)).long()
        count = extra + (torch.arange(L) < rows).long()
        count[0] += rows - int(count.sum())
        index = torch.repeat_interleave(torch.arange(L)[torch.randperm(L, generator=gen)], count)
        at = int(torch.randint(rows + 1, (1,), generator=gen))
        index = torch.cat([index[:at], torch.full((M - rows,), -1), index[at:]])
    else:
        index = torch.cat([index, torch.full((M - rows,), -1)])[torch.randperm(M, generator=gen)]
    return index.to(torch.int32)


def _normal(gen, shape, std):
    return torch.randn(shape, generator=gen, device="cuda") * std


def _activations(gen, M, K):
    """N(0, 1) with one channel in 200 twenty times as large, as the layers' inputs are."""
    x = _normal(gen, (M, K), 1.0)
    channels = torch.randperm(K, generator=gen, device="cuda")[:max(1, K // 200)]
    x[:, channels] *= 20.0
    return x.half()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    M, K = case["M"], case["K"]
    state = dict(case=case, x=_activations(gen, M, K))
    if case["op"] == "checkpoint":
        return state
    N, R, L = case["N"], case["R"], case["L"]
    state["a"] = _normal(gen, (L, R, K), K ** -0.5).half()
    state["b"] = _normal(gen, (L, N, R), 0.02).half()
    state["scaling"] = 2.0 ** -torch.randint(0, 3, (L,), generator=gen, device="cuda").float()
    index = _index(case, torch.Generator().manual_seed(seed))
    state["index"] = None if index is None else index.cuda()
    # the rows of every adapter, as a program that batches requests knows them
    state["rows"] = [(0, None)] if index is None else [
        (i, torch.nonzero(index == i).flatten().cuda()) for i in range(L) if bool((index == i).any())]
    if case["op"] != "backward":
        state["y"] = _normal(gen, (M, N), 1.5).half()
    if case["op"] != "forward":
        state["dy"] = _normal(gen, (M, N), 0.05).half()
        state["dx"] = _normal(gen, (M, K), 0.05).half()
    if case["op"] == "backward":
        h = torch.zeros((M, R), device="cuda")
        for i, rows in state["rows"]:
            at = slice(None) if rows is None else rows
            h[at] = state["x"][at].float() @ state["a"][i].float().t()
        state["h"] = h
        if case["group"]:
            q, s = _quantise(state["x"], case["group"])
            state["codes"] = (q + 128).to(torch.uint8).view(M, K)
            state["scales"] = s.view(M, K // case["group"])
            del state["x"]
    return state


# --- plain forms ------------------------------------------------------------------

def _quantise(x, group):
    """Whole numbers q (float32) and binary16 scales, both [M][groups][...]."""
    v = x.float().view(x.shape[0], -1, group)
    top = v.abs().amax(dim=2, keepdim=True)
    s = (top / 127).half()
    s = torch.where(s.float() * 127 < top, (s.view(torch.int16) + 1).view(torch.float16), s)
    s = torch.where(top == 0, torch.ones_like(s), s.clamp(max=515.5))
    q = torch.round(v / s.float()).clamp(-127, 127)
    return q, s


def _restore(q, s, shape):
    return (q * s.float()).half().view(shape)


def _forward(state):
    case = state["case"]
    out = state["y"].float()
    h = torch.zeros((case["M"], case["R"]), device=out.device)
    for i, rows in state["rows"]:
        at = slice(None) if rows is None else rows
        h_i = state["x"][at].float() @ state["a"][i].float().t()
        h[at] = h_i
        out[at] += state["scaling"][i] * (h_i @ state["b"][i].float().t())
    return out.half(), h


def _backward(state, x, h):
    dx = state["dx"].float()
    da = torch.zeros(state["a"].shape, device=dx.device)
    db = torch.zeros(state["b"].shape, device=dx.device)
    for i, rows in state["rows"]:
        at = slice(None) if rows is None else rows
        s = state["scaling"][i]
        dy = state["dy"][at].float()
        g = s * (dy @ state["b"][i].float())
        dx[at] += g @ state["a"][i].float()
        da[i] = g.t() @ x[at].float()
        db[i] = s * (dy.t() @ h[at])
    return dx.half(), da, db


def _plain(state):
    case = state["case"]
    if case["op"] == "forward":
        return _forward(state)[0]
    if case["op"] == "checkpoint":
        return _restore(*_quantise(state["x"], case["group"]), state["x"].shape)
    if case["op"] == "backward":
        if case["group"]:
            M, K = case["M"], case["K"]
            q = state["codes"].view(M, -1, case["group"]).float() - 128
            x = _restore(q, state["scales"].view(M, -1, 1), (M, K))
        else:
            x = state["x"]
        return _backward(state, x, state["h"])
    out, h = _forward(state)
    x = _restore(*_quantise(state["x"], case["group"]), state["x"].shape)
    return (out,) + _backward(state, x, h)


# --- the library's calls ----------------------------------------------------------

def _own(state):
    import w4a16_gemm_amd as w4
    case = state["case"]
    op = case["op"]
    if op == "forward":
        return w4.w4a16_lora_forward(state["y"], state["x"], state["a"], state["b"], state["index"], state["scaling"])
    if op == "checkpoint":
        codes, scales = w4.w4a16_act_quantize(state["x"], case["group"])
        return w4.w4a16_act_dequantize(codes, scales, case["group"])
    adapters = (state["a"], state["b"])
    if op == "backward":
        if case["group"]:
            return w4.w4a16_lora_backward_q8(state["dy"], state["codes"], state["scales"], case["group"], *adapters,
                                             state["h"], state["index"], state["scaling"], dx=state["dx"])
        return w4.w4a16_lora_backward(state["dy"], state["x"], *adapters, state["h"], state["index"],
                                      state["scaling"], dx=state["dx"])
    h = torch.empty((case["M"], case["R"]), dtype=torch.float32, device="cuda")
    out = w4.w4a16_lora_forward(state["y"], state["x"], *adapters, state["index"], state["scaling"], h=h)
    codes, scales = w4.w4a16_act_quantize(state["x"], case["group"])
    return (out,) + tuple(w4.w4a16_lora_backward_q8(state["dy"], codes, scales, case["group"], *adapters, h,
                                                    state["index"], state["scaling"], dx=state["dx"]))


def run(state):
    return _own(state) if own else _plain(state)


# --- the definitions in 64 bits ---------------------------------------------------

def _exact_values(x, group):
    """q S of every value, unrounded: the scale from the exponent of max|x| / 127."""
    v = x.double().reshape(-1, group)
    least = v.abs().max(dim=1).values / 127
    _, exponent = torch.frexp(least)                     # least = f 2^exponent, f in [1/2, 1)
    power = (exponent.long() - 11).clamp(min=-24)        # of two: the step between binary16 values there
    step = ((power + 1023) << 52).view(torch.float64)
    s = (torch.ceil(least / step) * step).clamp(max=515.5)
    s = torch.where(least == 0, torch.ones_like(s), s)[:, None]
    return ((v / s).round() * s).reshape(x.shape)


def _owner(state):
    M = state["case"]["M"]
    index = state["index"]
    return torch.zeros(M, dtype=torch.long, device="cuda") if index is None else index.long()


def _exact_h(state):
    owner = _owner(state)
    h = torch.zeros((state["case"]["M"], state["case"]["R"]), dtype=torch.float64, device="cuda")
    for i in range(state["case"]["L"]):
        mine = (owner == i).double()[:, None]
        h += mine * torch.mm(state["x"].double(), state["a"][i].double().t().contiguous())
    return h


def _exact_forward(state, h):
    owner = _owner(state)
    out = state["y"].double()
    for i in range(state["case"]["L"]):
        mine = (owner == i).double()[:, None]
        out.addmm_(mine * h, state["b"][i].double().t().contiguous(), alpha=float(state["scaling"][i]))
    return out


def _exact_backward(state, x, h):
    owner = _owner(state)
    dx = state["dx"].double()
    dy = state["dy"].double()
    da, db = [], []
    for i in range(state["case"]["L"]):
        s = float(state["scaling"][i])
        mine = (owner == i).double()[:, None]
        g = mine * torch.mm(dy, state["b"][i].double())
        dx.addmm_(g, state["a"][i].double(), alpha=s)
        da.append(s * torch.mm(g.t().contiguous(), x))
        db.append(s * torch.mm(dy.t().contiguous(), mine * h))
    return dx, torch.stack(da), torch.stack(db)


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "checkpoint":
        return _exact_values(state["x"], case["group"])
    if case["op"] == "forward":
        return _exact_forward(state, _exact_h(state))
    if case["op"] == "backward":
        if case["group"]:
            s = state["scales"].double().repeat_interleave(case["group"], dim=1)
            x = ((state["codes"].double() - 128) * s).half().double()
        else:
            x = state["x"].double()
        return _exact_backward(state, x, state["h"].double())
    h = _exact_h(state)
    x = _exact_values(state["x"], case["group"]).half().double()
    return (_exact_forward(state, h),) + _exact_backward(state, x, h)
