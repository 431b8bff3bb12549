"""Cases of the mixture-of-experts and vocabulary-head operators of the quantised layer:
routing of tokens to experts, products with the experts' packed weights and their
gradients, the weighted sum of the experts' outputs, and the softmax cross entropy over a
quantised vocabulary head.

``run`` makes one pass.  With ``own`` false it computes the operators in elementary torch
operations in 32 bits; with ``own`` true it calls the library.  ``exact`` computes the same
outputs in 64 bits from the definitions, with W^ = binary16((q - Z) S) the layer's weights:

  route     p = softmax(l[m]); the top_k largest, ties to the lowest index; their p, divided by
            their sum where renormalised; dl from the gradient of the weights
  experts   y[m][t] = W^_i x[m], i = index[m][t], 0 where i = -1
  backward  dx[m] = dx0[m] + sum_t W^_i^T dy[m][t]
  combine   out[m] = sum_t w[m][t] y[m][t]; dy[m][t] = w[m][t] dout[m]; dw[m][t] = <dout[m], y[m][t]>
  loss      l = W^ x[m]; lse = log sum exp l; loss = lse - l[target], 0 for rows without a
            target; dx[m] = dloss[m] (sum_v exp(l_v - lse) W^_v - W^_target)
"""

import math

import torch

own = False


def listed():
    """Layer shapes are those of the configurations and of the 1.5B-class model (1536, 8960,
    vocabulary 151936; 4096 -> 14336; 4096 -> 11008 at group 32 with act order)."""
    return [
        # decode, one sequence: the router's top 8 of 64, where only latency counts
        dict(name="route_token", op="route", M=1, E=64, T=8, bits=16, renorm=True, grad=False),
        # a training batch: probabilities as they are, with the gradient
        dict(name="route_train", op="route", M=8192, E=128, T=8, bits=32, renorm=False, grad=True),
        # decode, one sequence on two of eight large experts
        dict(name="experts_token", op="experts", M=1, T=2, E=8, K=4096, N=14336, bits=4, group=128, sym=False, act=False, pad=0.0),
        # decode of 24 sequences on small 8-bit experts, symmetric, a few rows for each
        dict(name="experts_batch", op="experts", M=24, T=4, E=32, K=1536, N=8960, bits=8, group=64, sym=True, act=False, pad=0.1),
        # prefill of a long prompt
        dict(name="experts_prefill", op="experts", M=4096, T=2, E=8, K=4096, N=14336, bits=4, group=128, sym=False, act=False, pad=0.0),
        # a ragged padded batch through act-order experts of group 32: gradient of their input
        dict(name="backward_ragged", op="backward", M=777, T=2, E=8, K=4096, N=11008, bits=4, group=32, sym=False, act=True, pad=0.1),
        # a training batch through 8-bit experts
        dict(name="backward_train", op="backward", M=4096, T=2, E=8, K=4096, N=14336, bits=8, group=128, sym=False, act=False, pad=0.0),
        # decode of 16 sequences: eight experts' outputs to one row each
        dict(name="combine_batch", op="combine", M=16, T=8, N=1536, grad=False),
        # a training batch, with the gradients
        dict(name="combine_train", op="combine", M=4096, T=4, N=4096, grad=True),
        # evaluation of a short continuation: the loss alone
        dict(name="loss_eval", op="loss", M=37, K=1536, V=151936, bits=4, group=128, sym=False, act=False, pad=0.0, grad=False),
        # fine-tuning on answers, prompt tokens without a target, 8-bit head: loss and gradient
        dict(name="loss_answers", op="loss", M=2048, K=1536, V=151936, bits=8, group=64, sym=False, act=False, pad=0.4, grad=True),
        # the largest: a long batch on a wide model
        dict(name="loss_train", op="loss", M=8192, K=4096, V=128000, bits=4, group=128, sym=False, act=False, pad=0.0, grad=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "experts", "experts", "backward", "backward", "combine", "loss", "loss"])
    if op == "route":
        E = _log_int(rng, 2, 512)
        return dict(op=op, M=_log_int(rng, 1, 16384), E=E, T=rng.randint(1, min(E, 16)), bits=rng.choice([16, 32]),
                    renorm=rng.random() < 0.5, grad=rng.random() < 0.5)
    if op == "combine":
        return dict(op=op, M=_log_int(rng, 1, 8192), T=rng.randint(1, 8), N=8 * _log_int(rng, 32, 1024), grad=rng.random() < 0.5)
    group = rng.choice([32, 64, 128, 0])
    K = 128 * _log_int(rng, 4, 64) if group else 64 * _log_int(rng, 8, 128)
    case = dict(op=op, M=_log_int(rng, 1, 8192), K=K, bits=rng.choice([4, 4, 8]), group=group or K, sym=rng.random() < 0.3,
                act=bool(group) and rng.random() < 0.25, pad=rng.choice([0.0, 0.1, 0.5]))
    if op == "loss":
        case.update(V=_log_int(rng, 1000, 160000), grad=rng.random() < 0.6)
    else:
        E = _log_int(rng, 1, 64)
        N = 16 * _log_int(rng, 32, 900)
        while E * K * N > 1 << 29:
            E = (E + 1) // 2
            N = 16 * (N // 32) if E == 1 else N
        case.update(T=rng.randint(1, min(E, 8)), E=E, N=N)
    most = _cost(listed()[-1])
    while _cost(case) > most:
        case["M"] = max(1, case["M"] // 2)
    return case


# --- work of one pass -------------------------------------------------------------

def _outputs(case):
    """Rows of the packed weights: a head's vocabulary is padded to whole words of zero points."""
    return case["N"] if "N" in case else -(-case["V"] // 16) * 16


def _layer_bytes(case):
    N, K, bits = _outputs(case), case["K"], case["bits"]
    G = K // case["group"]
    return N * K * bits // 8 + 2 * G * N + (0 if case["sym"] else G * N * bits // 8) + (4 * K if case["act"] else 0)


def _rows(case):
    return case["M"] - int(case["M"] * case["pad"])


def _cost(case):
    w = work(case)
    return w["bytes"] / 5e12 + w["flops"] / 5e14


def work(case):
    M, op = case["M"], case["op"]
    if op == "route":
        size = case["bits"] // 8
        n = {"bytes": M * case["E"] * size + 8 * M * case["T"], "flops": 4 * M * case["E"]}
        if case["grad"]:
            n = {"bytes": n["bytes"] + M * case["E"] * size + 4 * M * case["T"], "flops": 2 * n["flops"]}
        return n
    if op == "combine":
        T, N = case["T"], case["N"]
        n = {"bytes": 2 * M * T * N + 4 * M * T + 2 * M * N, "flops": 2 * M * T * N}
        if case["grad"]:
            n = {"bytes": n["bytes"] + 2 * M * N + 2 * M * T * N + 4 * M * T, "flops": 3 * n["flops"]}
        return n
    K, rows = case["K"], _rows(case)
    if op == "loss":
        one = 2 * rows * case["V"] * K
        if case["grad"]:
            return {"bytes": _layer_bytes(case) + 2 * rows * K + 2 * M * K + 16 * M, "flops": 3 * one}
        return {"bytes": _layer_bytes(case) + 2 * rows * K + 12 * M, "flops": one}
    T, N, E = case["T"], case["N"], case["E"]
    used = round(E * (1 - (1 - T / E) ** rows)) if E > T else E
    weights = used * _layer_bytes(case) + 4 * M * T
    if op == "experts":
        return {"bytes": weights + 2 * rows * K + 2 * M * T * N, "flops": 2 * rows * T * K * N}
    return {"bytes": weights + 4 * M * K + 2 * rows * T * N, "flops": 2 * rows * T * K * N}


# --- inputs -----------------------------------------------------------------------

def _normal(gen, shape, std=1.0):
    return torch.randn(shape, generator=gen, device="cuda") * std


def _activations(gen, M, K):
    """N(0, 1) with one channel in 200 twenty times as large, as the layers' inputs are."""
    x = _normal(gen, (M, K))
    channels = torch.randperm(K, generator=gen, device="cuda")[:max(1, K // 200)]
    x[:, channels] *= 20.0
    return x.half()


def _quantised(case, gen):
    """One layer's codes uint8 [N][K] (in stored order), scales [G][N], zero points [G][N] and
    stored order: round to nearest on N(0, 0.02) weights."""
    N, K, g = _outputs(case), case["K"], case["group"]
    w = _normal(gen, (N, K // g, g), 0.02)
    top = (1 << case["bits"]) - 1
    if case["sym"]:
        s = (w.abs().amax(2) / (top >> 1)).half()
        z = torch.full_like(s, (top + 1) // 2)
    else:
        lo = w.amin(2).clamp(max=0)
        s = ((w.amax(2).clamp(min=0) - lo) / top).half()
        z = torch.round(-lo / s.float()).clamp(0, top)
    q = (torch.round(w / s.float()[..., None]) + z.float()[..., None]).clamp(0, top)
    order = torch.randperm(K, generator=gen, device="cuda") if case["act"] else None
    return q.to(torch.uint8).view(N, K), s.t().contiguous(), z.t().contiguous().to(torch.uint8), order


def _packed(values, bits, places):
    """uint8 values [...][n] in 32-bit words: value e of a word in bits places[e] * bits and up."""
    per = 32 // bits
    v = values.view(*values.shape[:-1], -1, per).to(torch.int32)
    word = torch.zeros(v.shape[:-1], dtype=torch.int32, device=v.device)
    for e in range(per):
        word |= v[..., e] << (places[e] * bits)
    return word


# the weights' words hold their codes in this order, zero points theirs in plain order
ORDER = {4: (0, 4, 1, 5, 2, 6, 3, 7), 8: (0, 2, 1, 3)}


def _layers(case, seed, count):
    """The raw layers, and the generator that goes on to the other inputs."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return [_quantised(case, gen) for _ in range(count)], gen


def _pack_layers(case, layers):
    bits = case["bits"]
    words = []
    for q, _, _, order in layers:
        flat = _packed(q, bits, ORDER[bits]).flatten()
        words.append(flat if order is None else torch.cat([flat, order.to(torch.int32)]))
    plain = range(32 // bits)
    return dict(qweight=torch.stack(words), scales=torch.stack([s for _, s, _, _ in layers]),
                qzeros=None if case["sym"] else torch.stack([_packed(z, bits, plain) for _, _, z, _ in layers]),
                # group of every input channel: stored position p holds channel order[p]
                g_idx=torch.stack([torch.argsort(o).div(case["group"], rounding_mode="floor").to(torch.int32)
                                   for _, _, _, o in layers]) if case["act"] else None)


def _routing(case, gen):
    """Experts of every row, distinct and uneven, int32 [M][T]; the padding rows at the end have none."""
    M, E, T = case["M"], case["E"], case["T"]
    score = _normal(gen, (M, E)) + _normal(gen, (E,), 0.4)
    index = torch.topk(score, T, dim=1).indices.to(torch.int32)
    index[_rows(case):] = -1
    return index


def _inputs(case, seed):
    op, M = case["op"], case["M"]
    if op == "route":
        gen = torch.Generator(device="cuda").manual_seed(seed)
        logits = _normal(gen, (M, case["E"]), 2.0)
        state = dict(logits=logits.half() if case["bits"] == 16 else logits)
        if case["grad"]:
            state["dweights"] = _normal(gen, (M, case["T"]))
        return state, None
    if op == "combine":
        gen = torch.Generator(device="cuda").manual_seed(seed)
        T, N = case["T"], case["N"]
        weights = torch.rand((M, T), generator=gen, device="cuda")
        state = dict(y=_normal(gen, (M, T, N), 1.5).half(), weights=weights / weights.sum(1, keepdim=True))
        if case["grad"]:
            state["dout"] = _normal(gen, (M, N), 0.05).half()
        return state, None
    layers, gen = _layers(case, seed, case.get("E", 1))
    state = dict()
    if op == "loss":
        V, rows = case["V"], _rows(case)
        target = torch.randint(V, (M,), generator=gen, device="cuda")
        # rows from unsure to sure of their target, as a trained model's are
        sure = torch.rand((M, 1), generator=gen, device="cuda") * (1.5 * math.log(V) / (0.02 ** 2 * case["K"]))
        near = _values(case, layers[0], target)
        state["x"] = (_normal(gen, (M, case["K"])) + sure * near).half()
        none = torch.randperm(M, generator=gen, device="cuda")[:M - rows]
        target[none] = -100
        state["target"] = target.to(torch.int32)
        if case["grad"]:
            # mean over the rows with a target, times a loss scale of 1024
            state["dloss"] = torch.where(target >= 0, 1024.0 / max(rows, 1), 0.0).float()
        return state, layers
    state["index"] = _routing(case, gen)
    if op == "experts":
        state["x"] = _activations(gen, M, case["K"])
    else:
        state["dy"] = _normal(gen, (M, case["T"], case["N"]), 0.05).half()
        state["dx"] = _normal(gen, (M, case["K"]), 0.05).half()
    return state, layers


def _values(case, layer, rows):
    """Some rows of a layer's weights in 32 bits, in the channels' own order."""
    q, s, z, order = layer
    g = case["group"]
    w = (q[rows].view(len(rows), -1, g).float() - z.t()[rows].float()[..., None]) * s.t()[rows].float()[..., None]
    w = w.view(len(rows), -1)
    return w if order is None else w[:, torch.argsort(order)]


def prepare(case, seed):
    state, layers = _inputs(case, seed)
    if layers is not None:
        state.update(_pack_layers(case, layers))
    state["case"] = case
    return state


# --- plain forms ------------------------------------------------------------------

def _unpack(words, bits, places):
    shifts = torch.tensor([p * bits for p in places], dtype=torch.int32, device=words.device)
    return ((words[..., None] >> shifts) & ((1 << bits) - 1)).flatten(-2)


def _restore(state, used):
    """Weights float32 [U][N][K] in stored order, and the stored orders [U][K] or None."""
    case = state["case"]
    N, K, bits, g = _outputs(case), case["K"], case["bits"], case["group"]
    words = state["qweight"][used]
    codes = N * K * bits // 32
    q = _unpack(words[:, :codes], bits, ORDER[bits]).view(-1, N, K // g, g)
    if case["sym"]:
        z = 1 << (bits - 1)
    else:
        z = _unpack(state["qzeros"][used], bits, range(32 // bits)).transpose(1, 2)[..., None]
    w = (q - z).float() * state["scales"][used].float().transpose(1, 2)[..., None]
    return w.half().float().view(-1, N, K), words[:, codes:].long() if case["act"] else None


def _plan(index):
    """Used experts, and of every valid slot: the slot and its place in a padded [U][rows] batch."""
    slots = index.flatten().long()
    valid = torch.nonzero(slots >= 0).flatten()
    used, mine = torch.unique(slots[valid], return_inverse=True)
    order = torch.argsort(mine, stable=True)
    count = torch.bincount(mine, minlength=len(used))
    most = int(count.max())
    rank = torch.arange(len(order), device=order.device) - (torch.cumsum(count, 0) - count)[mine[order]]
    return used, valid[order], mine[order] * most + rank, most


def _padded(rows, place, U, most):
    batch = torch.zeros((U * most, rows.shape[1]), device=rows.device)
    batch[place] = rows
    return batch.view(U, most, -1)


def _experts(state):
    case = state["case"]
    M, T, N = case["M"], case["T"], case["N"]
    y = torch.zeros((M * T, N), device="cuda")
    used, slot, place, most = _plan(state["index"])
    w, order = _restore(state, used)
    x = _padded(state["x"][torch.div(slot, T, rounding_mode="floor")].float(), place, len(used), most)
    if order is not None:
        x = x.gather(2, order[:, None, :].expand_as(x))
    out = torch.bmm(w, x.transpose(1, 2).contiguous()).transpose(1, 2).reshape(-1, N)
    y[slot] = out[place]
    return y.half().view(M, T, N)


def _backward(state):
    case = state["case"]
    M, T, N, K = case["M"], case["T"], case["N"], case["K"]
    used, slot, place, most = _plan(state["index"])
    w, order = _restore(state, used)
    dy = _padded(state["dy"].view(M * T, N)[slot].float(), place, len(used), most)
    g = torch.bmm(dy, w)
    if order is not None:
        g = g.gather(2, torch.argsort(order, dim=1)[:, None, :].expand_as(g))
    part = torch.zeros((M * T, K), device="cuda")
    part[slot] = g.reshape(-1, K)[place]
    return (state["dx"].float() + part.view(M, T, K).sum(1)).half()


def _route(state):
    case = state["case"]
    l = state["logits"].float()
    e = torch.exp(l - l.amax(1, keepdim=True))
    p = e / e.sum(1, keepdim=True)
    index = torch.sort(l, dim=1, descending=True, stable=True).indices[:, :case["T"]]
    chosen = p.gather(1, index)
    w = chosen / chosen.sum(1, keepdim=True) if case["renorm"] else chosen
    if not case["grad"]:
        return index.to(torch.int32), w
    dw = state["dweights"]
    mean = (w * dw).sum(1, keepdim=True)
    if case["renorm"]:
        dl = torch.zeros_like(l).scatter_(1, index, w * (dw - mean))
    else:
        dl = (-p * mean).scatter_add_(1, index, w * dw)
    return index.to(torch.int32), w, dl.to(state["logits"].dtype)


def _combine(state):
    y, w = state["y"].float(), state["weights"]
    out = (w[..., None] * y).sum(1).half()
    if not state["case"]["grad"]:
        return out
    d = state["dout"].float()[:, None, :]
    return out, (w[..., None] * d).half(), (d * y).sum(2)


def _loss(state):
    case = state["case"]
    w, order = _restore(state, torch.zeros(1, dtype=torch.long, device="cuda"))
    w = w[0, :case["V"]]
    # rows without a target take no part
    rows = torch.nonzero(state["target"] >= 0).flatten()
    target = state["target"][rows].long()
    x = state["x"][rows].float()
    if order is not None:
        x = x[:, order[0]]
    l = x @ w.t()
    top = l.amax(1, keepdim=True)
    e = torch.exp(l - top)
    total = e.sum(1, keepdim=True)
    lse = torch.zeros(case["M"], device="cuda")
    lse[rows] = (top + torch.log(total)).flatten()
    loss = torch.zeros_like(lse)
    loss[rows] = lse[rows] - l.gather(1, target[:, None]).flatten()
    if not case["grad"]:
        return loss, lse
    p = e / total
    p[torch.arange(len(rows), device="cuda"), target] -= 1
    g = state["dloss"][rows, None] * (p @ w)
    if order is not None:
        g = g[:, torch.argsort(order[0])]
    dx = torch.zeros((case["M"], case["K"]), device="cuda")
    dx[rows] = g
    return loss, lse, dx.half()


def _plain(state):
    op = state["case"]["op"]
    return {"route": _route, "experts": _experts, "backward": _backward, "combine": _combine, "loss": _loss}[op](state)


# --- the library's calls ----------------------------------------------------------

def _own(state):
    import w4a16_gemm_amd as w4
    case = state["case"]
    op = case["op"]
    if op == "route":
        index, weights = w4.w4a16_route(state["logits"], case["T"], renormalise=case["renorm"])
        if not case["grad"]:
            return index, weights
        return index, weights, w4.w4a16_route_backward(state["dweights"], state["logits"], index, weights,
                                                       renormalise=case["renorm"])
    if op == "combine":
        out = w4.w4a16_experts_combine(state["y"], state["weights"])
        if not case["grad"]:
            return out
        return (out,) + tuple(w4.w4a16_experts_combine_backward(state["dout"], state["y"], state["weights"]))
    four = case["bits"] == 4
    experts = (state["qweight"], state["scales"], state["qzeros"], state["g_idx"], case["group"])
    if op == "experts":
        gemm = w4.w4a16_experts_gemm if four else w4.w8a16_experts_gemm
        return gemm(state["x"], *experts, state["index"])
    if op == "backward":
        backward = w4.w4a16_experts_backward if four else w4.w8a16_experts_backward
        return backward(state["dy"], *experts, state["index"], case["K"], dx=state["dx"])
    head = (state["qweight"][0], state["scales"][0], None if case["sym"] else state["qzeros"][0],
            state["g_idx"][0] if case["act"] else None, case["group"])
    forward = w4.w4a16_head_loss if four else w4.w8a16_head_loss
    loss, lse = forward(state["x"], *head, state["target"], vocab=case["V"])
    if not case["grad"]:
        return loss, lse
    backward = w4.w4a16_head_loss_backward if four else w4.w8a16_head_loss_backward
    return loss, lse, backward(state["dloss"], state["x"], *head, state["target"], lse, vocab=case["V"])


def run(state):
    return _own(state) if own else _plain(state)


# --- the definitions in 64 bits ---------------------------------------------------

def _exact_weights(case, layer):
    """binary16((q - Z) S) of one layer, float64 [N][K] in the channels' own order."""
    q, s, z, order = layer
    at = torch.arange(case["K"], device="cuda") // case["group"]
    w = ((q.double() - z.double()[at].t()) * s.double()[at].t()).half().double()
    if order is None:
        return w
    out = torch.empty_like(w)
    out[:, order] = w
    return out


def _exact_route(case, state):
    l = state["logits"].double()
    p = torch.softmax(l, dim=1)
    # the largest first, of equal ones the lowest index: E - index breaks the ties of the ranks
    rank = torch.unique(l, return_inverse=True)[1] * case["E"] + torch.arange(case["E"] - 1, -1, -1, device="cuda")
    index = torch.topk(rank, case["T"], dim=1).indices
    w = p.gather(1, index)
    total = w.sum(1, keepdim=True) if case["renorm"] else 1.0
    if not case["grad"]:
        return index.to(torch.int32), w / total
    # the chain rule through w = c / total and p: dp of the chosen, then the softmax
    dw = state["dweights"].double()
    dc = (dw - (dw * w / total).sum(1, keepdim=True)) / total if case["renorm"] else dw
    dp = torch.zeros_like(p).scatter_(1, index, dc)
    return index.to(torch.int32), w / total, p * (dp - (p * dp).sum(1, keepdim=True))


def _exact_loss(case, state, w):
    w = w[:case["V"]]
    M, K = case["M"], case["K"]
    lse = torch.zeros(M, dtype=torch.float64, device="cuda")
    loss = torch.zeros_like(lse)
    dx = torch.zeros((M, K), dtype=torch.float64, device="cuda")
    wt = w.t().contiguous()
    rows = torch.nonzero(state["target"] >= 0).flatten()
    for at in rows.split(1024):
        target = state["target"][at].long()
        l = torch.mm(state["x"][at].double(), wt)
        lse[at] = torch.logsumexp(l, dim=1)
        loss[at] = lse[at] - l[torch.arange(len(at), device="cuda"), target]
        if case["grad"]:
            p = torch.exp_(l.sub_(lse[at][:, None]))
            dx[at] = state["dloss"][at].double()[:, None] * (torch.mm(p, w) - w[target])
    return (loss, lse, dx) if case["grad"] else (loss, lse)


def exact(case, seed):
    state, layers = _inputs(case, seed)
    op, M = case["op"], case["M"]
    if op == "route":
        return _exact_route(case, state)
    if op == "combine":
        y, w = state["y"].double(), state["weights"].double()
        out = torch.matmul(w[:, None, :], y)[:, 0]
        if not case["grad"]:
            return out
        d = state["dout"].double()
        return out, w[:, :, None] * d[:, None, :], torch.matmul(y, d[:, :, None])[..., 0]
    if op == "loss":
        return _exact_loss(case, state, _exact_weights(case, layers[0]))
    T = case["T"]
    index = state["index"].flatten()
    if op == "experts":
        y = torch.zeros((M * T, case["N"]), dtype=torch.float64, device="cuda")
        for i, layer in enumerate(layers):
            at = torch.nonzero(index == i).flatten()
            y[at] = torch.mm(state["x"][at // T].double(), _exact_weights(case, layer).t().contiguous())
        return y.view(M, T, case["N"])
    dx = state["dx"].double()
    dy = state["dy"].view(M * T, case["N"])
    for i, layer in enumerate(layers):
        at = torch.nonzero(index == i).flatten()
        dx[at // T] += torch.mm(dy[at].double(), _exact_weights(case, layer))   # an expert has a row once at most
    return dx
