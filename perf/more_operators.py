"""The experts' linear layers in bf16, as measured work: forward, and backward to the rows and to the weights.

A case names one operator in "op":

* "linear": each expert's bf16 weight matrix times the bf16 rows it received, packed or padded, with an optional bias, gated activation
  and residual, and optionally the rows before the activation, which training keeps.
* "rows": the gradient of the rows: each expert's matrix, from the other side, times the rows' output gradients, optionally carried on
  through the gated activation that made those rows.
* "weights": the gradient of every expert's matrix (and bias), summed over the expert's rows, in bf16 or float32.

With "E" 0 a case is a dense layer, as a shared expert is: every row meets the one matrix.

`run` computes them in elementary torch operations, or, where `own` is true, by the library's calls."""

import math

import torch

own = False


def listed():
    return [
        # a single sequence's next token: eight experts' gate and up matrices are read for it
        dict(name="linear_one_token", op="linear", T=1, E=256, K=8, H=7168, N=4096, gated=True, bias=False, residual=False, save=False, padded=False, zipf=0.0),
        # a decoding step of 128 sequences in the padded layout, with the experts' biases
        dict(name="linear_decode", op="linear", T=128, E=256, K=8, H=7168, N=4096, gated=True, bias=True, residual=False, save=False, padded=True, zipf=0.0),
        # a training batch's first layer, which keeps the rows before the activation for the backward pass
        dict(name="linear_train", op="linear", T=4096, E=256, K=8, H=7168, N=4096, gated=True, bias=False, residual=False, save=True, padded=False, zipf=0.0),
        # the largest batch the library is benchmarked on
        dict(name="linear_large", op="linear", T=32768, E=256, K=8, H=7168, N=4096, gated=True, bias=False, residual=False, save=False, padded=False, zipf=0.0),
        # the shared expert's second layer in a decoding step: the combined experts' output is its residual; latency is all there is
        dict(name="shared_decode", op="linear", T=7, E=0, K=1, H=2048, N=7168, gated=False, bias=False, residual=True, save=False, padded=False, zipf=0.0),
        # the same for a prefill batch, with a bias
        dict(name="shared_prefill", op="linear", T=4096, E=0, K=1, H=2048, N=7168, gated=False, bias=True, residual=True, save=False, padded=False, zipf=0.0),
        # a training batch, from the second layer's output gradients through it and the activation
        dict(name="rows_gated", op="rows", T=4096, E=256, K=8, H=2048, N=7168, gated=True, padded=False, zipf=0.0),
        # and on through the first layer to the received rows, a few popular experts
        dict(name="rows_first", op="rows", T=4096, E=256, K=8, H=7168, N=4096, gated=False, padded=False, zipf=1.2),
        # the tiny model of the tests
        dict(name="rows_tiny", op="rows", T=64, E=16, K=2, H=256, N=256, gated=True, padded=False, zipf=0.0),
        # one of eight GPUs' experts, first layer, gradients in the weights' type
        dict(name="weights_first", op="weights", T=4096, E=32, K=8, H=7168, N=4096, dtype="bfloat16", bias=False, padded=False, zipf=0.0),
        # their second layer with popular experts, float32 gradients as an optimizer accumulates them, and the biases'
        dict(name="weights_second", op="weights", T=4093, E=32, K=8, H=2048, N=7168, dtype="float32", bias=True, padded=False, zipf=1.2),
        # the shared expert of a large batch
        dict(name="weights_shared", op="weights", T=32768, E=0, K=1, H=2048, N=7168, dtype="bfloat16", bias=True, padded=False, zipf=0.0),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["linear", "linear", "rows", "weights"])
    E = 0 if rng.random() < 0.25 else log(2, 16 if op == "weights" else 64)
    case = dict(op=op, T=log(1, 4096), E=E, K=min(max(E, 1), log(1, 8)), H=8 * log(8, 896), N=16 * log(4, 448),
                padded=E > 0 and rng.random() < 0.25, zipf=rng.choice([0.0, 1.2]))
    if op == "weights":
        return dict(case, dtype=rng.choice(["bfloat16", "float32"]), bias=rng.random() < 0.5)
    case["gated"] = rng.random() < 0.5
    if op == "linear":
        case.update(bias=rng.random() < 0.5, residual=rng.random() < 0.3, save=case["gated"] and rng.random() < 0.4)
    return case


def work(case):
    T, E, K, H, N = (case[k] for k in ("T", "E", "K", "H", "N"))
    R = T * K
    hit = E * (1 - (1 - K / E) ** T) if E else 1  # matrices with a row, for even routing
    flops = 2 * R * N * H
    if case["op"] == "linear":
        out = N // 2 if case["gated"] else N
        each = 2 * H + 2 * out + (2 * out if case["residual"] else 0) + (2 * N if case["save"] else 0)
        return {"bytes": hit * N * (2 * H + (2 if case["bias"] else 0)) + R * each, "flops": flops}
    if case["op"] == "rows":
        return {"bytes": hit * N * 2 * H + R * (2 * N + (8 * H if case["gated"] else 2 * H)), "flops": flops}
    size = 2 if case["dtype"] == "bfloat16" else 4
    return {"bytes": R * 2 * (N + H) + max(E, 1) * N * (H + (1 if case["bias"] else 0)) * size, "flops": flops}


# ---- inputs --------------------------------------------------------------------------------------------------------------------


def _ids(case, g):
    """K different experts for each token, evenly or by Zipf popularity."""
    T, E = case["T"], case["E"]
    key = -torch.log(-torch.log(torch.rand(T, E, generator=g, device="cuda").clamp(1e-20, 1 - 1e-7)))
    if case["zipf"]:
        rank = torch.randperm(E, generator=g, device="cuda").float() + 1
        key = key - case["zipf"] * torch.log(rank)
    return key.topk(case["K"], dim=1).indices


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    T, E, K, H, N = (case[k] for k in ("T", "E", "K", "H", "N"))

    def rows(n, width, spread):
        """bf16 rows, with channels of unequal size where activations have them."""
        size = torch.exp(0.5 * torch.randn(width, generator=g, device="cuda")) if spread else 1.0
        x = torch.empty(n, width, dtype=torch.bfloat16, device="cuda")
        for part in x.split(65536):
            part.copy_(torch.randn(part.shape, generator=g, device="cuda") * size)
        return x

    state = {"case": case}
    if E:
        counts = torch.bincount(_ids(case, g).flatten(), minlength=E)
        state["counts"] = counts.to(torch.int32)
        state["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
        counts = counts.tolist()
    else:
        counts = [T]
    R = E * T if case["padded"] else T * K  # padded: a capacity of T rows for each expert, so that nothing is dropped
    first, spans = 0, []
    for e, n in enumerate(counts):  # the rows of each expert that has any
        if n:
            spans.append((e, e * T if case["padded"] else first, n))
        first += n
    state["spans"], state["rows"] = spans, R
    if case["op"] != "weights":
        state["w"] = torch.empty(max(E, 1), N, H, dtype=torch.bfloat16, device="cuda")
        for w in state["w"]:
            w.copy_(torch.randn(N, H, generator=g, device="cuda") / math.sqrt(H if case["op"] == "linear" else N))
    if case["op"] == "linear":
        state["a"] = rows(R, H, True)
        out = N // 2 if case["gated"] else N
        state["bias"] = (0.1 * torch.randn(max(E, 1), N, generator=g, device="cuda")).to(torch.bfloat16) if case["bias"] else None
        state["residual"] = rows(R, out, False) if case["residual"] else None
        if case["padded"]:  # rows of no expert stay as they are
            state["y"] = torch.zeros(R, out, dtype=torch.bfloat16, device="cuda")
            state["p"] = torch.zeros(R, N, dtype=torch.bfloat16, device="cuda") if case["save"] else None
        return state
    state["grad"] = rows(R, N, False)
    if case["op"] == "rows":
        state["p"] = rows(R, 2 * H, True) if case["gated"] else None
        if case["padded"]:
            state["grad_a"] = torch.zeros(R, 2 * H if case["gated"] else H, dtype=torch.bfloat16, device="cuda")
    else:
        state["a"] = rows(R, H, True)
    return state


# ---- the plain forms -----------------------------------------------------------------------------------------------------------


def _linear(case, s):
    N, half = case["N"], case["N"] // 2
    y = torch.zeros(s["rows"], half if case["gated"] else N, dtype=torch.bfloat16, device="cuda")
    kept = torch.zeros(s["rows"], N, dtype=torch.bfloat16, device="cuda") if case["save"] else None
    for e, first, n in s["spans"]:
        at = slice(first, first + n)
        p = s["a"][at].float() @ s["w"][e].float().T
        if case["bias"]:
            p += s["bias"][e].float()
        if case["save"]:
            kept[at] = p.to(torch.bfloat16)
        if case["gated"]:
            gate, up = p[:, :half], p[:, half:]
            p = gate / (1 + torch.exp(-gate)) * up
        if case["residual"]:
            p = p + s["residual"][at].float()
        y[at] = p.to(torch.bfloat16)
    return {"y": y, "p": kept} if case["save"] else y


def _rows(case, s):
    H = case["H"]
    grad_a = torch.zeros(s["rows"], 2 * H if case["gated"] else H, dtype=torch.bfloat16, device="cuda")
    for e, first, n in s["spans"]:
        at = slice(first, first + n)
        d = s["grad"][at].float() @ s["w"][e].float()
        if case["gated"]:
            gate, up = s["p"][at].float().split(H, 1)
            f = 1 / (1 + torch.exp(-gate))
            d = torch.cat([d * up * (f * (1 + gate * (1 - f))), d * (gate * f)], 1)
        grad_a[at] = d.to(torch.bfloat16)
    return grad_a


def _weights(case, s):
    E, N, H = max(case["E"], 1), case["N"], case["H"]
    dtype = getattr(torch, case["dtype"])
    grad_w = torch.zeros(E, N, H, dtype=dtype, device="cuda")
    grad_b = torch.zeros(E, N, dtype=dtype, device="cuda") if case["bias"] else None
    for e, first, n in s["spans"]:
        g = s["grad"][first:first + n].float()
        grad_w[e] = (g.T @ s["a"][first:first + n].float()).to(dtype)
        if case["bias"]:
            grad_b[e] = g.sum(0).to(dtype)
    return {"w": grad_w, "b": grad_b} if case["bias"] else grad_w


def run(state):
    case = state["case"]
    if own:
        return _own(case, state)
    return {"linear": _linear, "rows": _rows, "weights": _weights}[case["op"]](case, state)


def _own(case, s):
    import combine_ep_dispatch_amd as ep

    if case["padded"]:  # into buffers that the program keeps, as its expert rows
        if case["op"] == "linear":
            ep.ep_expert_linear(s["a"], s["w"], s["counts"], case["T"], ep.EP_ACT_SWIGLU if case["gated"] else ep.EP_ACT_NONE, s["y"],
                                bias=s["bias"], residual=s["residual"], p=s["p"])
            return {"y": s["y"], "p": s["p"]} if case["save"] else s["y"]
        if case["op"] == "rows":
            ep.ep_expert_linear_backward(s["grad"], s["w"], s["counts"], case["T"], s["grad_a"], p=s["p"])
            return s["grad_a"]
        handle = ep.PaddedHandle(s["counts"], None, None, case["E"], case["T"])
    else:
        handle = ep.Handle(s["counts"], s["offsets"], None, None, case["E"]) if case["E"] else None
    if case["op"] == "linear":
        out = ep.expert_linear(s["a"], s["w"], handle, bias=s["bias"], activation=ep.EP_ACT_SWIGLU if case["gated"] else ep.EP_ACT_NONE,
                               residual=s["residual"], save=case["save"])
        return {"y": out[0], "p": out[1]} if case["save"] else out
    if case["op"] == "rows":
        return ep.expert_linear_backward(s["grad"], s["w"], handle, p=s["p"])
    out = ep.expert_linear_backward_weights(s["grad"], s["a"], handle, dtype=getattr(torch, case["dtype"]), bias=case["bias"])
    return {"w": out[0], "b": out[1]} if case["bias"] else out


# ---- the definition in 64 bits -------------------------------------------------------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    N, H, R = case["N"], case["H"], s["rows"]

    def zeros(*shape):
        return torch.zeros(shape, dtype=torch.float64, device="cuda")

    if case["op"] == "linear":
        y, kept = zeros(R, N // 2 if case["gated"] else N), zeros(R, N) if case["save"] else None
        for e, first, n in s["spans"]:
            p = torch.mm(s["a"][first:first + n].double(), s["w"][e].double().t())
            if s["bias"] is not None:
                p = p + s["bias"][e].double()
            if case["save"]:
                kept[first:first + n] = p
            if case["gated"]:
                p = p[:, : N // 2] * torch.sigmoid(p[:, : N // 2]) * p[:, N // 2:]
            y[first:first + n] = p if s["residual"] is None else p + s["residual"][first:first + n].double()
        return {"y": y, "p": kept} if case["save"] else y
    if case["op"] == "rows":
        grad = zeros(R, 2 * H if case["gated"] else H)
        for e, first, n in s["spans"]:
            d = torch.mm(s["w"][e].double().t(), s["grad"][first:first + n].double().t()).t()
            if case["gated"]:
                u, v = s["p"][first:first + n, :H].double(), s["p"][first:first + n, H:].double()
                f, rest = torch.sigmoid(u), torch.sigmoid(-u)
                grad[first:first + n, :H] = d * v * (f + u * f * rest)
                grad[first:first + n, H:] = d * u * f
            else:
                grad[first:first + n] = d
        return grad
    grad_w, grad_b = zeros(max(case["E"], 1), N, H), zeros(max(case["E"], 1), N)
    for e, first, n in s["spans"]:
        g = s["grad"][first:first + n].double()
        grad_w[e] = torch.mm(s["a"][first:first + n].double().t(), g).t()
        grad_b[e] = torch.mm(g.new_ones(1, n), g)[0]
    return {"w": grad_w, "b": grad_b} if case["bias"] else grad_w
