"""Plain 64-bit statements of routing, quantised rows and the experts'
products (test infrastructure only; shares no code with the GPU path).

The rules are those of ep_route, ep_route_backward, ep_quantize_rows,
ep_dequantize_rows and ep_expert_product in include/ep.h.  MXFP4 follows the
OCP microscaling formats specification v1.0: E2M1 elements (0, 0.5, 1, 1.5,
2, 3, 4, 6 and their negatives), one E8M0 scale (2^(b-127), 255 = NaN) per
32 elements, the scale's exponent floor(log2(amax)) - 2.
"""

import numpy as np

from .codecs import bf16_bits_to_f32, e4m3_to_f32

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
SOFTMAX, SIGMOID = 0, 1


# ---- routing ----------------------------------------------------------------

def clean_logits(logits):
    """NaN counts as -inf, +inf as the largest finite binary32."""
    z = np.asarray(logits, dtype=np.float64)
    z = np.where(np.isnan(z), -np.inf, z)
    return np.minimum(z, float(np.finfo(np.float32).max))


def scores(z, score):
    on = ~np.isneginf(z)
    if score == SIGMOID:
        with np.errstate(over="ignore"):
            return np.where(on, 1.0 / (1.0 + np.exp(-z)), 0.0)
    m = np.where(on.any(axis=1, keepdims=True), z.max(axis=1, keepdims=True), 0.0)
    p = np.where(on, np.exp(z - m), 0.0)
    total = p.sum(axis=1, keepdims=True)
    return np.where(total > 0, p / np.where(total > 0, total, 1.0), 0.0)


def _ratio(z, ids, score):
    """s_k / sum_j s_j over the entries with ids >= 0, without underflow:
    each s is taken relative to exp(min(max z, 0))."""
    on = ids >= 0
    zk = np.where(on, np.take_along_axis(z, np.maximum(ids, 0), axis=1), -np.inf)
    m = np.where(on.any(axis=1), zk.max(axis=1), 0.0)[:, None]
    with np.errstate(over="ignore", invalid="ignore"):
        if score == SIGMOID:
            u = np.exp(np.minimum(zk, 0.0) - np.minimum(m, 0.0)) / (1.0 + np.exp(-np.abs(zk)))
        else:
            u = np.exp(zk - m)
    u = np.where(on, u, 0.0)
    total = u.sum(axis=1, keepdims=True)
    return u / np.where(total > 0, total, 1.0)


def group_score(best):
    """The sum of a group's one or two largest v, rounded to 40 binary places
    below the larger magnitude."""
    total, m = sum(best), max(abs(v) for v in best)
    if m == 0 or np.isinf(m):
        return total
    q = 41 - int(np.frexp(m)[1])  # m = f * 2^e with 0.5 <= f < 1
    return float(np.ldexp(np.rint(np.ldexp(total, q)), -q))


def route(logits, top_k, bias=None, n_group=1, topk_group=1, score=SIGMOID, renormalize=True, scale=1.0):
    """-> (ids int32 [T, K], weights float64 [T, K]); one token at a time."""
    z = clean_logits(logits)
    T, E = z.shape
    s = scores(z, score)
    if bias is not None:  # (steers the choice only: s is the logits')
        b = np.asarray(bias, dtype=np.float64)
        z = np.where(np.isnan(b) | np.isneginf(b), -np.inf, z)
    ids = np.full((T, top_k), -1, dtype=np.int32)
    for t in range(T):
        v = s[t] + (b if bias is not None else 0.0)
        on = ~np.isneginf(z[t])
        if n_group > 1:
            n = E // n_group
            rank = []
            for g in range(n_group):
                best = sorted((float(v[e]) for e in range(g * n, g * n + n) if on[e]), reverse=True)[:2]
                if best:
                    rank.append((-group_score(best), g))
            kept = {g for _, g in sorted(rank)[:topk_group]}
            on = on & np.array([e // n in kept for e in range(E)])
        key = v if bias is not None else z[t]
        order = sorted((e for e in range(E) if on[e]), key=lambda e: (-key[e], e))[:top_k]
        ids[t, :len(order)] = order
    on = ids >= 0
    if renormalize:
        w = _ratio(z, ids, score)
    else:
        w = np.where(on, np.take_along_axis(s, np.maximum(ids, 0), axis=1), 0.0)
    return ids, scale * w


def _entries(z, ids):
    """Ids that count: inside [0, E) and of an expert that is on; else -1."""
    ids = np.asarray(ids, dtype=np.int64)
    E = z.shape[1]
    ok = (ids >= 0) & (ids < E)
    zk = np.take_along_axis(z, np.where(ok, ids, 0), axis=1)
    return np.where(ok & ~np.isneginf(zk), ids, -1)


def route_weights(logits, ids, score, renormalize, scale):
    """The weights of given ids as a function of the logits (what
    route_backward differentiates)."""
    z = clean_logits(logits)
    ids = _entries(z, ids)
    if renormalize:
        return scale * _ratio(z, ids, score)
    s = scores(z, score)
    return scale * np.where(ids >= 0, np.take_along_axis(s, np.maximum(ids, 0), axis=1), 0.0)


def route_backward(grad_w, logits, ids, score, renormalize, scale):
    """-> (grad float64 [T, E], magnitude [T, E]): the gradient, and the sum
    of the magnitudes of the terms it is made of (for error bounds)."""
    z = clean_logits(logits)
    ids = _entries(z, ids)
    on = ids >= 0
    g = np.where(on, np.asarray(grad_w, dtype=np.float64), 0.0)
    at = np.maximum(ids, 0)
    zk = np.where(on, np.take_along_axis(z, at, axis=1), 0.0)
    grad, mag = np.zeros_like(z), np.zeros_like(z)
    rows = np.broadcast_to(np.arange(z.shape[0])[:, None], ids.shape)
    if score == SIGMOID:
        e = np.exp(-np.abs(zk))
        rest = np.where(zk > 0, e, 1.0) / (1.0 + e)  # 1 - s
        slope = e / (1.0 + e) ** 2  # s (1 - s)
    if renormalize:
        q = _ratio(z, ids, score)
        f = scale * q * (rest if score == SIGMOID else 1.0)
        np.add.at(grad, (rows, at), np.where(on, f * (g - (g * q).sum(axis=1, keepdims=True)), 0.0))
        np.add.at(mag, (rows, at), np.where(on, abs(f) * (abs(g) + (abs(g) * q).sum(axis=1, keepdims=True)), 0.0))
    elif score == SIGMOID:
        np.add.at(grad, (rows, at), np.where(on, scale * g * slope, 0.0))
        np.add.at(mag, (rows, at), np.where(on, abs(scale * g * slope), 0.0))
    else:
        p = scores(z, SOFTMAX)
        pk = np.where(on, np.take_along_axis(p, at, axis=1), 0.0)
        np.add.at(grad, (rows, at), scale * g)
        np.add.at(mag, (rows, at), abs(scale * g))
        grad = p * (grad - (scale * g * pk).sum(axis=1, keepdims=True))
        mag = p * (mag + (abs(scale * g) * pk).sum(axis=1, keepdims=True))
    return grad, mag


# ---- rows in MXFP4 -----------------------------------------------------------

def quantize_mxfp4(x_bits):
    """BF16 bits [R, H] -> (codes uint8 [R, H/2], scales uint8 [R, H/32])."""
    x = bf16_bits_to_f32(x_bits).astype(np.float64)
    R, H = x.shape
    b = x.reshape(R, H // 32, 32)
    bad = ~np.isfinite(b).all(axis=2)
    a = np.abs(np.where(np.isfinite(b), b, 0.0))
    top = a.max(axis=2)
    _, e = np.frexp(np.where(top > 0, top, 4.0))  # top = m * 2^e with 0.5 <= m < 1
    e = np.maximum(e.astype(np.int64) - 3, -127)
    v = a / np.exp2(e.astype(np.float64))[:, :, None]
    code = np.zeros(v.shape, dtype=np.int64)
    for c in range(1, 8):  # the next value from the midpoint on; the midpoint itself where c is even
        mid = (E2M1[c - 1] + E2M1[c]) / 2
        code = np.where((v > mid) | ((v == mid) & (c % 2 == 0)), c, code)
    code = np.where(bad[:, :, None], 0, code | (np.signbit(b).astype(np.int64) << 3)).reshape(R, H)
    scale = np.where(bad, 255, e + 127)
    return (code[:, 0::2] | (code[:, 1::2] << 4)).astype(np.uint8), scale.astype(np.uint8)


def mxfp4_values(q, scale):
    """Codes and scales -> float64 values."""
    q, scale = np.asarray(q), np.asarray(scale)
    code = np.stack([q & 15, q >> 4], axis=-1).reshape(q.shape[:-1] + (-1,)).astype(np.int64)
    v = np.where(code & 8, -1.0, 1.0) * E2M1[code & 7]
    s = np.where(scale == 255, np.nan, np.exp2(scale.astype(np.float64) - 127))
    return v * np.repeat(s, 32, axis=-1)


def fp8_values(q, scale):
    """E4M3 codes and one binary32 scale per 128 channels -> float64 values."""
    return e4m3_to_f32(q).astype(np.float64) * np.repeat(np.asarray(scale, dtype=np.float64), 128, axis=-1)


# ---- the experts' products ---------------------------------------------------

def expert_product(a, w, spans, gated):
    """a float64 [R, H], w float64 [E, N, H], spans [(first, count)] -> (y
    float64 [R, O] with NaN in rows of no expert, absolute error scale [R,
    O]): y before its rounding to BF16, and the sum over h of |w a| carried
    through the activation's slopes."""
    R, N = a.shape[0], w.shape[1]
    O = N // 2 if gated else N
    y, mag = np.full((R, O), np.nan), np.full((R, O), np.nan)
    for e, (first, count) in enumerate(spans):
        if count == 0:
            continue
        rows = a[first:first + count]
        p, m = rows @ w[e].T, np.abs(rows) @ np.abs(w[e]).T
        if gated:
            g, u = p[:, :O], p[:, O:]
            with np.errstate(over="ignore"):
                sg = 1.0 / (1.0 + np.exp(-g))
            silu = g * sg
            # |silu'| <= 1.1 everywhere
            y[first:first + count] = silu * u
            mag[first:first + count] = 1.1 * m[:, :O] * (np.abs(u) + m[:, O:] * 2.0 ** -8) + np.abs(silu) * m[:, O:]
        else:
            y[first:first + count], mag[first:first + count] = p, m
    return y, mag
