"""An expert layer trained in bf16 as a user runs it: route, dispatch in
EP_RECV_BF16, the experts' two layers, the shared expert's with the combined
rows as its residual; and the whole backward pass.  Each step is compared with
the oracle on the GPU's own inputs to that step, so that a step's rounding is
not carried into the next comparison; one gradient of the whole is compared
with differences of the loss in 64 bits."""

import numpy as np
import pytest
import torch

from oracle import operators as ops
from tests.gpu_run import host

pytestmark = pytest.mark.gpu


def values(t):
    torch.cuda.synchronize()
    return t.double().cpu().numpy()


def close(got, want, bound, mine=None):
    v = values(got).reshape(want.shape)
    mine = np.ones(len(v), dtype=bool) if mine is None else mine
    ok = np.abs(v - want) <= bound + 2.0 ** -8 * (np.abs(want) + bound) + 2.0 ** -133
    assert ok[mine].all(), "%d off" % (~ok[mine]).sum()


@pytest.mark.parametrize("T,padded", [(1, False), (96, True), (700, False)])
def test_training_step(gpu, T, padded):
    ep = gpu
    E, K, H, I = 16, 4, 256, 192
    g = torch.Generator(device="cuda")
    g.manual_seed(T)
    new = lambda *shape: torch.randn(*shape, generator=g, device="cuda").bfloat16()
    x, logits, go = new(T, H), torch.randn(T, E, generator=g, device="cuda"), new(T, H)
    w1, b1, w2, b2 = new(E, 2 * I, H) / 16, new(E, 2 * I) / 8, new(E, H, I) / 16, new(E, H) / 8
    s1, s2 = new(2 * I, H) / 16, new(H, I) / 16  # the shared expert

    ids, tw = ep.route(logits, K)
    if padded:
        rx, _, count, h = ep.low_latency_dispatch(x, ids, T, E, format=ep.EP_RECV_BF16)
        spans = [(e * T, int(n)) for e, n in enumerate(host(count))]
    else:
        rx, _, _, h = ep.dispatch(x, ids, tw, E, format=ep.EP_RECV_BF16)
        off = host(h.expert_offset)
        spans = [(int(off[e]), int(off[e + 1] - off[e])) for e in range(E)]
    R = rx.numel() // H
    mine = np.zeros(R, dtype=bool)
    for first, n in spans:
        mine[first:first + n] = True

    def rows(t):
        v = values(t).reshape(R, -1)
        return np.where(mine[:, None], v, 0.0)  # unused rows hold anything

    mid, p = ep.expert_linear(rx, w1, h, b1, ep.EP_ACT_SWIGLU, save=True)
    want = ops.expert_linear(rows(rx), values(w1), values(b1), None, spans, True)
    close(mid, *want["y"], mine)
    close(p, *want["p"], mine)
    y = ep.expert_linear(mid, w2, h, b2)
    close(y, *ops.expert_linear(rows(mid), values(w2), values(b2), None, spans, False)["y"], mine)
    out = ep.low_latency_combine(y, h, tw) if padded else ep.combine(y, h, tw)
    smid, sp = ep.expert_linear(x, s1, None, activation=ep.EP_ACT_SWIGLU, save=True)
    total = ep.expert_linear(smid, s2, None, residual=out)
    close(total, *ops.expert_linear(values(smid), values(s2)[None], None, values(out), [(0, T)], False)["y"])

    # backward: the residual's gradient is the output's
    flat = lambda t: t.reshape(R, -1)
    grad_y, grad_tw = ep.combine_backward(go, flat(y), h, tw)
    grad_y = grad_y.view_as(y)
    assert bool((grad_y.reshape(R, -1)[torch.from_numpy(~mine).cuda()] == 0).all())
    grad_p = ep.expert_linear_backward(grad_y, w2, h, p=p)
    close(grad_p, *ops.expert_linear_backward(rows(grad_y), values(w2), rows(p), spans), mine)
    for gy, a, n in ((grad_y, mid, H), (grad_p, rx, 2 * I)):
        gw, gb = ep.expert_linear_backward_weights(gy, a, h, bias=True)
        want = ops.expert_linear_backward_weights(rows(gy), rows(a), spans)
        close(gw, *want["w"])
        close(gb, *want["b"])
    grad_r = ep.expert_linear_backward(grad_p, w1, h)
    close(grad_r, *ops.expert_linear_backward(rows(grad_p), values(w1), None, spans), mine)
    grad_x = ep.dispatch_backward(flat(grad_r), h)
    assert grad_x.shape == (T, H) and bool(torch.isfinite(grad_x).all())
    grad_sp = ep.expert_linear_backward(go, s2, None, p=sp)
    close(grad_sp, *ops.expert_linear_backward(values(go), values(s2)[None], values(sp), [(0, T)]))
    acc = torch.zeros(1, H, I, device="cuda")
    for _ in range(2):  # two microbatches into one float32 gradient
        ep.ep_expert_linear_backward_weights(go, smid, None, 0, acc, accumulate=True)
    want, bound = ops.expert_linear_backward_weights(values(go), values(smid), [(0, T)])["w"]
    assert np.all(np.abs(values(acc) - 2 * want) <= 2 * bound + 2.0 ** -22 * np.abs(want))


def test_gradient_of_the_whole_layer(gpu):
    """The loss's slope along one direction of every weight, from the gradients
    that the calls give, against a central difference in 64 bits.  Each bf16
    rounding on the way (rows between the layers, their gradients, the
    gradients themselves) moves a term by at most 2^-8 of it; five of them,
    summed over magnitudes."""
    ep = gpu
    T, E, K, H, I = 24, 4, 2, 64, 48
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    new = lambda *shape: torch.randn(*shape, generator=g, device="cuda").bfloat16()
    x, go, logits = new(T, H), new(T, H), torch.randn(T, E, generator=g, device="cuda")
    w1, w2 = new(E, 2 * I, H) / 8, new(E, H, I) / 8
    ids, tw = ep.route(logits, K)
    rx, _, _, h = ep.dispatch(x, ids, tw, E, format=ep.EP_RECV_BF16)
    mid, p = ep.expert_linear(rx, w1, h, activation=ep.EP_ACT_SWIGLU, save=True)
    y = ep.expert_linear(mid, w2, h)
    grad_y, _ = ep.combine_backward(go, y, h, tw)
    grad_p = ep.expert_linear_backward(grad_y, w2, h, p=p)
    g1 = values(ep.expert_linear_backward_weights(grad_p, rx, h, torch.float32))
    g2 = values(ep.expert_linear_backward_weights(grad_y, mid, h, torch.float32))
    off = host(h.expert_offset)
    spans = [(int(off[e]), int(off[e + 1] - off[e])) for e in range(E)]
    up = np.zeros((T * K, H))  # the loss's gradient of every expert row, exact
    np.add.at(up, host(h.slot).ravel(), np.repeat(values(go), K, 0) * values(tw).ravel()[:, None])

    def loss(v1, v2):
        m = ops.expert_linear(values(rx), v1, None, None, spans, True)["y"][0]
        return (up * ops.expert_linear(m, v2, None, None, spans, False)["y"][0]).sum()

    v1, v2 = values(w1), values(w2)
    rng = np.random.default_rng(0)
    d1, d2 = rng.standard_normal(v1.shape), rng.standard_normal(v2.shape)
    step = 1e-5
    slope1 = (loss(v1 + step * d1, v2) - loss(v1 - step * d1, v2)) / (2 * step)
    slope2 = (loss(v1, v2 + step * d2) - loss(v1, v2 - step * d2)) / (2 * step)
    # magnitudes of what the gradients are summed from
    m2 = ops.expert_linear_backward_weights(np.abs(up), np.abs(values(mid)), spans)["w"][0]
    dmid = np.zeros((T * K, I))
    for e, (first, n) in enumerate(spans):
        dmid[first:first + n] = np.abs(up[first:first + n]) @ np.abs(v2[e])
    pv = values(p)
    gate, lin = np.abs(pv[:, :I]), np.abs(pv[:, I:])
    mp = np.concatenate([dmid * lin * (1 + gate), dmid * gate], 1)  # slopes of silu at most 1 + |g|, its value at most |g|
    m1 = ops.expert_linear_backward_weights(mp, np.abs(values(rx)), spans)["w"][0]
    assert abs((g2 * d2).sum() - slope2) <= 5 * 2.0 ** -8 * (m2 * np.abs(d2)).sum()
    assert abs((g1 * d1).sum() - slope1) <= 5 * 2.0 ** -8 * (m1 * np.abs(d1)).sum()
