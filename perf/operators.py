"""The operators around the dispatch and combine of an MoE layer, as measured work: routing (and its gradient), rows held in
microscaled 4-bit or in 8-bit floating point, and the experts' products on those rows.

A case names one operator in "op":

* "route": router scores to expert ids and weights (group-limited or plain top-k); "route_backward": its gradient.
* "quantize": rows to 4-bit (one power-of-two scale per 32 channels) or E4M3 (one binary32 scale per 128), and the values they stand for.
* "dispatch": tokens sorted by expert into such rows, with the routing layout and the routed weights.
* "product": each expert's weight matrix (4-bit) times the rows of that expert, packed or padded, with or without the gated activation.

`run` computes them in elementary torch operations, or, where `own` is true, by the library's calls."""

import math

import numpy as np
import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # one decoding step of 128 sequences: latency is all there is; the selection carries a balancing bias
        dict(name="route_decode", op="route", T=128, E=256, K=8, groups=8, kept=4, score="sigmoid", bias=True, renorm=True, scale=2.5, dtype="float32", masked=0),
        # a long prefill batch, scores in the model's own bf16
        dict(name="route_prefill", op="route", T=32768, E=256, K=8, groups=8, kept=4, score="sigmoid", bias=False, renorm=True, scale=1.0, dtype="bfloat16", masked=0),
        # a training batch: the gradient of the weights, back to the scores
        dict(name="route_backward", op="route_backward", T=32768, E=256, K=8, groups=8, kept=4, score="sigmoid", bias=False, renorm=True, scale=2.5, dtype="float32", masked=0),
        # a decoding step's tokens to their experts in 4 bits
        dict(name="dispatch_decode", op="dispatch", format="mxfp4", T=128, H=7168, E=256, K=8, zipf=0.0),
        # prefill with a few popular experts
        dict(name="dispatch_prefill", op="dispatch", format="mxfp4", T=4096, H=7168, E=256, K=8, zipf=1.2),
        # the activations between an expert's two products: odd row count, as routing gives it
        dict(name="quantize_rows", op="quantize", format="mxfp4", rows=32747, H=2048),
        # the weight matrices of 16 experts, once, when a model is loaded
        dict(name="quantize_weights", op="quantize", format="mxfp4", rows=65536, H=7168),
        # a single sequence's next token: eight experts' weights are read for it
        dict(name="product_one_token", op="product", format="mxfp4", T=1, E=256, K=8, H=7168, N=4096, gated=True, padded=False, zipf=0.0),
        # a decoding step in the padded layout, rows as the 8-bit dispatch leaves them
        dict(name="product_decode", op="product", format="fp8", T=128, E=256, K=8, H=7168, N=4096, gated=True, padded=True, zipf=0.0),
        # prefill, first product (gate and up together)
        dict(name="product_prefill", op="product", format="mxfp4", T=4096, E=256, K=8, H=7168, N=4096, gated=True, padded=False, zipf=0.0),
        # prefill, second product, 8-bit rows, popular experts
        dict(name="product_down", op="product", format="fp8", T=4096, E=256, K=8, H=2048, N=7168, gated=False, padded=False, zipf=1.2),
        # the largest batch the library is benchmarked on
        dict(name="product_large", op="product", format="mxfp4", T=32768, E=256, K=8, H=7168, N=4096, gated=True, padded=False, zipf=0.0),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["route", "route_backward", "dispatch", "quantize", "product", "product"])
    if op in ("route", "route_backward"):
        groups = rng.choice([1, 1, 2, 4, 8])
        E = groups * max(2, log(16, 512) // groups)
        kept = rng.randint(1, groups)
        K = min(log(1, 16), kept * (E // groups))
        score = rng.choice(["sigmoid", "softmax"])
        renorm = rng.random() < 0.7
        if op == "route_backward" and renorm:
            K = max(K, 2)  # a single renormalised weight is a constant
        masked = rng.choice([0, 0, E // 8]) if kept * (E // groups) >= K + E // 8 else 0
        return dict(op=op, T=log(1, 32768), E=E, K=K, groups=groups, kept=kept, score=score, bias=op == "route" and rng.random() < 0.5, renorm=renorm,
                    scale=rng.choice([1.0, 2.5]), dtype=rng.choice(["float32", "bfloat16"]), masked=masked)
    form = rng.choice(["mxfp4", "mxfp4", "fp8"])
    unit = 32 if form == "mxfp4" else 128
    if op == "quantize":
        return dict(op=op, format=form, rows=log(1, 65536), H=unit * max(1, log(128, 7168) // unit))
    E = log(4, 256)
    K = min(E, log(1, 8))
    if op == "dispatch":
        return dict(op=op, format=form, T=log(1, 4096), H=unit * max(1, log(256, 7168) // unit), E=E, K=K, zipf=rng.choice([0.0, 1.2]))
    gated = rng.random() < 0.5
    E = log(4, 64)
    K = min(E, log(1, 8))
    return dict(op=op, format=form, T=log(1, 4096), E=E, K=K, H=128 * max(1, log(256, 7168) // 128), N=16 * max(1, log(128, 7168) // 16), gated=gated,
                padded=rng.random() < 0.3, zipf=rng.choice([0.0, 1.2]))


def _row_bytes(case):
    """Bytes of one row of H channels with its scales."""
    return case["H"] // 2 + case["H"] // 32 if case["format"] == "mxfp4" else case["H"] + case["H"] // 32


def work(case):
    if case["op"] in ("route", "route_backward"):
        T, E, K, size = case["T"], case["E"], case["K"], 4 if case["dtype"] == "float32" else 2
        both = 2 if case["op"] == "route_backward" else 1  # the scores are read, and the gradient is written
        return {"bytes": both * T * E * size + 8 * T * K, "flops": 8 * T * E}
    if case["op"] == "quantize":
        row = _row_bytes(case)
        return {"bytes": case["rows"] * (4 * case["H"] + 2 * row), "flops": 4 * case["rows"] * case["H"]}
    if case["op"] == "dispatch":
        T, H, K, row = case["T"], case["H"], case["K"], _row_bytes(case)
        return {"bytes": T * (2 * H + 16 * K) + T * K * (2 * row + 2 * H + 4), "flops": 4 * T * H}
    T, E, K, H, N = (case[k] for k in ("T", "E", "K", "H", "N"))
    hit = E * (1 - (1 - K / E) ** T)  # experts with a row, for even routing
    out = N // 2 if case["gated"] else N
    return {"bytes": hit * N * (H // 2 + H // 32) + T * K * (_row_bytes(case) + 2 * out), "flops": 2 * T * K * N * H}


# ---- inputs --------------------------------------------------------------------------------------------------------------------


def _e2m1(a):
    """Magnitudes up to 6 to the nearest of E2M1's, ties to the even code."""
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    return torch.round(a / step) * step


def _mxfp4(x):
    """Blocks of 32 channels: the values (as multiples of the scale) and the scales' exponents."""
    b = x.float().unflatten(-1, (-1, 32))
    top = b.abs().amax(-1, keepdim=True)
    e = torch.where(top > 0, torch.frexp(top).exponent - 3, 0).clamp(-127, 127)
    s = torch.ldexp(torch.ones_like(top), e)
    return (torch.sign(b) * _e2m1((b.abs() / s).clamp(max=6.0))), e


def _pack(v, e):
    """E2M1 values and exponents to bytes: two codes a byte, the even channel in the low half, and one biased exponent per block."""
    grid = torch.tensor(E2M1, device=v.device)
    code = torch.bucketize(v.abs().flatten(-2), grid).to(torch.uint8) | (torch.signbit(v.flatten(-2)).to(torch.uint8) << 3)
    return code[..., 0::2] | (code[..., 1::2] << 4), (e.squeeze(-1) + 127).to(torch.uint8)


def _fp8(x):
    b = x.float().unflatten(-1, (-1, 128))
    top = b.abs().amax(-1, keepdim=True)
    s = torch.where(top > 0, (top / 448.0).clamp(min=2.0 ** -126), 1.0)
    return (b / s).clamp(-448.0, 448.0).to(torch.float8_e4m3fn), s


def _ids(case, g):
    """K different experts for each token, evenly or by Zipf popularity."""
    T, E = case["T"], case["E"]
    key = -torch.log(-torch.log(torch.rand(T, E, generator=g, device="cuda").clamp(1e-20, 1 - 1e-7)))
    if case["zipf"]:
        rank = torch.randperm(E, generator=g, device="cuda").float() + 1
        key = key - case["zipf"] * torch.log(rank)
    return key.topk(case["K"], dim=1).indices.to(torch.int32)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    state = {"case": case}
    if case["op"] in ("route", "route_backward"):
        T, E, K = case["T"], case["E"], case["K"]
        z = normal(T, E)
        if case["masked"]:  # experts that are switched off
            z[:, torch.randperm(E, generator=g, device="cuda")[: case["masked"]]] = -math.inf
        state["logits"] = z.to(getattr(torch, case["dtype"]))
        state["bias"] = 0.1 * normal(E) if case["bias"] else None
        if case["op"] == "route_backward":
            state["ids"] = _route(case, state["logits"], None)[0]
            state["grad_w"] = normal(T, K)
        return state
    if case["op"] == "quantize":
        # channels of unequal size, as activations have them
        state["x"] = (normal(case["rows"], case["H"]) * torch.exp(0.5 * normal(case["H"]))).to(torch.bfloat16)
        return state
    T, E, K, H = case["T"], case["E"], case["K"], case["H"]
    ids = _ids(case, g)
    if case["op"] == "dispatch":
        state["ids"], state["x"] = ids, (normal(T, H) * torch.exp(0.5 * normal(H))).to(torch.bfloat16)
        state["weights"] = torch.rand(T, K, generator=g, device="cuda")
        return state
    N = case["N"]
    counts = torch.bincount(ids.flatten().long(), minlength=E)
    state["most"] = int(counts.max())  # rows of the fullest expert
    state["counts"] = counts.to(torch.int32)
    state["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
    rows = E * T if case["padded"] else T * K  # padded: a capacity of T rows for each expert, so that nothing is dropped
    q, s = [], []
    for r in range(0, rows, 65536):
        x = (normal(min(65536, rows - r), H) * torch.exp(0.5 * normal(H))).to(torch.bfloat16)
        v, e = _mxfp4(x) if case["format"] == "mxfp4" else _fp8(x)
        v, e = _pack(v, e) if case["format"] == "mxfp4" else (v.flatten(-2).view(torch.uint8), e.squeeze(-1))
        q.append(v)
        s.append(e)
    state["a"], state["a_scale"] = torch.cat(q), torch.cat(s)
    state["w"] = torch.empty(E, N, H // 2, dtype=torch.uint8, device="cuda")
    state["w_scale"] = torch.empty(E, N, H // 32, dtype=torch.uint8, device="cuda")
    for e in range(E):
        state["w"][e], state["w_scale"][e] = _pack(*_mxfp4(normal(N, H) / math.sqrt(H)))
    # rows of no expert stay as they are
    state["y"] = torch.zeros(rows, N // 2 if case["gated"] else N, dtype=torch.bfloat16, device="cuda")
    return state


# ---- the plain forms -----------------------------------------------------------------------------------------------------------


def _route(case, logits, bias):
    """In 64 bits, so that scores next to each other keep their order."""
    T, E, K, G = case["T"], case["E"], case["K"], case["groups"]
    z = logits.double()
    off = torch.isneginf(z)
    s = 1 / (1 + torch.exp(-z)) if case["score"] == "sigmoid" else torch.exp(z - z.amax(1, keepdim=True))
    if case["score"] == "softmax":
        s = s / s.sum(1, keepdim=True)
    v = (s if bias is None else s + bias.double()).masked_fill(off, -math.inf)
    key = (z if bias is None else v).masked_fill(off, -math.inf)
    if G > 1:
        best = v.view(T, G, E // G).sort(dim=2, descending=True).values[:, :, :2]
        score = torch.round(best.masked_fill(torch.isneginf(best), 0).sum(2) * 2.0 ** 40)  # sums nearer than that are tied
        score = score.masked_fill(torch.isneginf(best[:, :, 0]), -math.inf)
        keep = torch.zeros(T, G, dtype=torch.bool, device=z.device)
        keep.scatter_(1, score.sort(dim=1, descending=True, stable=True).indices[:, : case["kept"]], True)
        key = key.masked_fill(~keep.repeat_interleave(E // G, 1), -math.inf)
    top = key.sort(dim=1, descending=True, stable=True)
    none = torch.isneginf(top.values[:, :K])
    ids = top.indices[:, :K]
    w = s.gather(1, ids).masked_fill(none, 0)
    if case["renorm"]:
        w = w / w.sum(1, keepdim=True).clamp(min=1e-300)
    return ids.masked_fill(none, -1).to(torch.int32), (w * case["scale"]).float()


def _route_backward(case, logits, ids, grad_w):
    z = logits.double()
    none = ids < 0
    at = ids.clamp(min=0).long()
    g = grad_w.double().masked_fill(none, 0)
    c = case["scale"]
    if case["score"] == "sigmoid":
        s = 1 / (1 + torch.exp(-z.gather(1, at)))
        s = s.masked_fill(none, 0)
        if case["renorm"]:
            w = s / s.sum(1, keepdim=True).clamp(min=1e-300)
            d = c * w * (1 - s) * (g - (g * w).sum(1, keepdim=True))
        else:
            d = c * g * s * (1 - s)
        return torch.zeros_like(z).scatter_add_(1, at, d).to(logits.dtype)
    p = torch.exp(z - z.amax(1, keepdim=True))
    p = p / p.sum(1, keepdim=True)
    w = p.gather(1, at).masked_fill(none, 0)
    if case["renorm"]:
        w = w / w.sum(1, keepdim=True).clamp(min=1e-300)
        d = c * w * (g - (g * w).sum(1, keepdim=True))
        return torch.zeros_like(z).scatter_add_(1, at, d).to(logits.dtype)
    up = torch.zeros_like(z).scatter_add_(1, at, c * g)
    return (p * (up - (c * g * w).sum(1, keepdim=True))).to(logits.dtype)


def _values(x, form):
    """What the rows stand for after quantisation, in bf16."""
    v, s = _mxfp4(x) if form == "mxfp4" else _fp8(x)
    return (torch.ldexp(v, s) if form == "mxfp4" else v.float() * s).flatten(-2).to(torch.bfloat16)


def _decode(q, scale, form):
    """Bytes and scales to binary32 values."""
    if form == "fp8":
        return (q.view(torch.float8_e4m3fn).float().unflatten(-1, (-1, 128)) * scale.unsqueeze(-1)).flatten(-2)
    half = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=q.device)
    pair = torch.stack([half.repeat(16), half.repeat_interleave(16)], 1)  # byte -> (low, high)
    v = pair[q.int()].flatten(-2).unflatten(-1, (-1, 32))
    return v.mul_(torch.ldexp(torch.ones(1, device=q.device), scale.int() - 127).unsqueeze(-1)).flatten(-2)


def _dispatch(case, x, ids, weights):
    order = ids.flatten().sort(stable=True).indices  # by expert, then by (token, k)
    slot = torch.empty_like(order).scatter_(0, order, torch.arange(order.numel(), device=order.device))
    values = _values(x, case["format"])[order // case["K"]]
    return {"values": values, "slot": slot.view_as(ids).to(torch.int32), "weight": weights.flatten()[order]}


def _product(case, s):
    most, rows = s["most"], s["a"].shape[0]
    at = torch.arange(most, device=s["a"].device)
    if case["padded"]:
        row = torch.arange(case["E"], device=at.device)[:, None] * case["T"] + at
        there = at < s["counts"][:, None]
    else:
        row = s["offsets"][:-1, None] + at
        there = row < s["offsets"][1:, None]
    a = _decode(s["a"], s["a_scale"], case["format"])[row.clamp(max=rows - 1)]
    y = torch.bmm(a, _decode(s["w"], s["w_scale"], "mxfp4").transpose(1, 2))
    if case["gated"]:
        gate, up = y.chunk(2, -1)
        y = gate / (1 + torch.exp(-gate)) * up
    out = torch.zeros(rows + 1, y.shape[-1], dtype=torch.bfloat16, device=y.device)  # the last row takes what no row asks for
    out[torch.where(there, row, rows)] = y.to(torch.bfloat16)
    return out[:rows]


def run(state):
    case, s = state["case"], state
    if own:
        return _own(case, s)
    if case["op"] == "route":
        ids, w = _route(case, s["logits"], s["bias"])
        return {"ids": ids, "weights": w}
    if case["op"] == "route_backward":
        return _route_backward(case, s["logits"], s["ids"], s["grad_w"])
    if case["op"] == "quantize":
        return _values(s["x"], case["format"])
    if case["op"] == "dispatch":
        return _dispatch(case, s["x"], s["ids"], s["weights"])
    return _product(case, s)


def _own(case, s):
    import combine_ep_dispatch_amd as ep

    if case["op"] in ("route", "route_backward"):
        score = ep.EP_SCORE_SIGMOID if case["score"] == "sigmoid" else ep.EP_SCORE_SOFTMAX
        if case["op"] == "route":
            ids, w = ep.route(s["logits"], case["K"], bias=s["bias"], n_group=case["groups"], topk_group=case["kept"], score=score, renormalize=case["renorm"], scale=case["scale"])
            return {"ids": ids, "weights": w}
        return ep.route_backward(s["grad_w"], s["logits"], s["ids"], score=score, renormalize=case["renorm"], scale=case["scale"])
    form = ep.EP_RECV_MXFP4_G32 if case["format"] == "mxfp4" else ep.EP_RECV_FP8_E4M3_G128
    if case["op"] == "quantize":
        return ep.dequantize_rows(*ep.quantize_rows(s["x"], form), form)
    if case["op"] == "dispatch":
        recv, scale, weight, handle = ep.dispatch(s["x"], s["ids"], s["weights"], case["E"], format=form)
        return {"values": ep.dequantize_rows(recv, scale, form), "slot": handle.slot, "weight": weight}
    act = ep.EP_ACT_SWIGLU if case["gated"] else ep.EP_ACT_NONE
    if case["padded"]:
        ep.ep_expert_product(s["a"], s["a_scale"], form, s["w"], s["w_scale"], s["counts"], case["T"], act, s["y"])
    else:
        ep.ep_expert_product(s["a"], s["a_scale"], form, s["w"], s["w_scale"], s["offsets"], 0, act, s["y"])
    return s["y"]


# ---- the definition in 64 bits -------------------------------------------------------------------------------------------------


def _exact_route(case, z, bias):
    T, E, K = case["T"], case["E"], case["K"]
    z = z.double().cpu().numpy()
    off = np.isneginf(z)
    with np.errstate(over="ignore"):
        if case["score"] == "sigmoid":
            s = 1.0 / (1.0 + np.exp(-z))
        else:
            s = np.exp(z - z.max(axis=1, keepdims=True))
            s /= s.sum(axis=1, keepdims=True)
    v = s if bias is None else s + bias.double().cpu().numpy()
    ok = ~off
    if case["groups"] > 1:
        n = E // case["groups"]
        two = np.sort(np.where(off, -np.inf, v).reshape(T, -1, n), axis=2)[:, :, -2:]
        gs = np.rint(np.where(np.isneginf(two), 0.0, two).sum(axis=2) * 2.0 ** 40)
        gs[np.isneginf(two[:, :, -1])] = -np.inf
        place = np.argsort(np.argsort(-gs, axis=1, kind="stable"), axis=1, kind="stable")
        ok &= np.repeat(place < case["kept"], n, axis=1)
    order = np.argsort(np.where(ok, -(z if bias is None else v), np.inf), axis=1, kind="stable")[:, :K]
    there = np.take_along_axis(ok, order, axis=1)
    w = np.where(there, np.take_along_axis(s, order, axis=1), 0.0)
    if case["renorm"]:
        w = w / np.maximum(w.sum(axis=1, keepdims=True), 1e-300)
    return torch.from_numpy(w * case["scale"])


def _exact_route_backward(case, z, ids, g):
    z, ids, g = z.double().cpu().numpy(), ids.cpu().numpy(), g.double().cpu().numpy()
    there = ids >= 0
    g = np.where(there, g, 0.0)
    hot = (ids[:, :, None] == np.arange(case["E"])) & there[:, :, None] if ids.size * case["E"] <= 1 << 27 else None
    if hot is None:
        grad, rows = np.zeros_like(z), 4096
        for t in range(0, z.shape[0], rows):
            part = dict(case, T=min(rows, z.shape[0] - t))
            grad[t:t + rows] = _exact_route_backward(part, torch.from_numpy(z[t:t + rows]), torch.from_numpy(ids[t:t + rows]), torch.from_numpy(g[t:t + rows])).numpy()
        return torch.from_numpy(grad)
    chosen = hot.any(axis=1)
    up = (g[:, :, None] * hot).sum(axis=1)  # dL/dw, at the chosen expert's place
    if case["score"] == "sigmoid":
        f = 1.0 / (1.0 + np.exp(-z))
        slope = f * (1.0 / (1.0 + np.exp(z)))
    else:
        f = np.exp(z - z.max(axis=1, keepdims=True))
        slope = None
    # w = scale * f / total, total over the chosen (renormalised), over all (softmax) or 1
    if case["renorm"]:
        total = (f * chosen).sum(axis=1, keepdims=True)
        df = case["scale"] * (up / total - (up * f).sum(axis=1, keepdims=True) / total ** 2) * chosen
    elif case["score"] == "softmax":
        total = f.sum(axis=1, keepdims=True)
        df = case["scale"] * (up / total - (up * f).sum(axis=1, keepdims=True) / total ** 2)
    else:
        df = case["scale"] * up
    return torch.from_numpy(df * (f if slope is None else slope))


def _exact_values(x, form):
    x = x.double()
    if form == "fp8":
        b = x.unflatten(-1, (-1, 128))
        top = b.abs().amax(-1, keepdim=True)
        s = torch.where(top > 0, (top / 448).float().double().clamp(min=2.0 ** -126), 1.0)
        a = (b / s).float().double().abs()  # the quotient is a binary32 value by definition
        quantum = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** -6))) - 3)
        return (torch.sign(b) * torch.round(a / quantum) * quantum * s).flatten(-2)
    b = x.unflatten(-1, (-1, 32))
    top = b.abs().amax(-1, keepdim=True)
    s = torch.exp2(torch.floor(torch.log2(torch.where(top > 0, top, 4.0))).clamp(min=-125) - 2)
    a = b.abs() / s
    value = torch.zeros_like(a)
    for low, high in zip(E2M1[:-1], E2M1[1:]):
        middle = (low + high) / 2
        up = a >= middle if E2M1.index(high) % 2 == 0 else a > middle
        value = torch.where(up, high, value)
    return (torch.sign(b) * value * s).flatten(-2)


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "route":
        return {"ids": None, "weights": _exact_route(case, state["logits"], state["bias"])}
    if case["op"] == "route_backward":
        return _exact_route_backward(case, state["logits"], state["ids"], state["grad_w"])
    if case["op"] == "quantize":
        return torch.cat([_exact_values(x, case["format"]) for x in state["x"].split(4096)])
    if case["op"] == "dispatch":
        flat = state["ids"].flatten().cpu().numpy()
        order = torch.from_numpy(np.argsort(flat, kind="stable")).cuda()
        values = _exact_values(state["x"], case["format"])
        return {"values": values[torch.div(order, case["K"], rounding_mode="floor")], "slot": None, "weight": state["weights"].double().flatten()[order]}
    grid = torch.tensor(E2M1, dtype=torch.float64, device="cuda")

    def four(q, scale):
        code = torch.stack([q & 15, q >> 4], -1).flatten(-2).int()
        v = grid[code & 7] * (1 - 2 * (code >> 3))
        return v * torch.exp2(scale.double() - 127).repeat_interleave(32, -1)

    counts, y = state["counts"].tolist(), torch.zeros(state["y"].shape, dtype=torch.float64, device="cuda")
    first = 0
    for e, n in enumerate(counts):
        r = e * case["T"] if case["padded"] else first
        first += n
        if n == 0:
            continue
        q, scale = state["a"][r:r + n], state["a_scale"][r:r + n]
        a = four(q, scale) if case["format"] == "mxfp4" else q.view(torch.float8_e4m3fn).double() * scale.double().repeat_interleave(128, -1)
        p = a @ four(state["w"][e], state["w_scale"][e]).T
        if case["gated"]:
            p = p[:, : case["N"] // 2] * torch.sigmoid(p[:, : case["N"] // 2]) * p[:, case["N"] // 2:]
        y[r:r + n] = p
    return y
