"""The whole expert layer as a user runs it: route, dispatch, the experts'
two products with the rows requantised between them, combine; and the
training direction back to the router's logits.  Each step is compared with
the oracle on the GPU's own inputs to that step, so that a step's rounding
is not carried into the next comparison."""

import numpy as np
import pytest
import torch

import oracle
from oracle import operators as ops
from tests.gpu_run import host
from tests.test_expert_product_gpu import check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["mxfp4", "fp8"])
@pytest.mark.parametrize("T,padded", [(1, False), (96, True), (700, False)])
def test_expert_layer(gpu, fmt, T, padded):
    ep = gpu
    E, K, H, I = 32, 4, 512, 256
    form = ep.EP_RECV_MXFP4_G32 if fmt == "mxfp4" else ep.EP_RECV_FP8_E4M3_G128
    values = ops.mxfp4_values if fmt == "mxfp4" else ops.fp8_values
    g = torch.Generator(device="cuda")
    g.manual_seed(T)
    x = torch.randn(T, H, generator=g, device="cuda").bfloat16()
    logits = torch.randn(T, E, generator=g, device="cuda")
    w1, s1 = ep.quantize_rows(0.05 * torch.randn(E * 2 * I, H, generator=g, device="cuda").bfloat16())
    w2, s2 = ep.quantize_rows(0.05 * torch.randn(E * H, I, generator=g, device="cuda").bfloat16())
    w1, s1, w2, s2 = w1.view(E, 2 * I, -1), s1.view(E, 2 * I, -1), w2.view(E, H, -1), s2.view(E, H, -1)

    ids, tw = ep.route(logits, K, n_group=4, topk_group=2)
    want_ids, _ = ops.route(logits.double().cpu().numpy(), K, n_group=4, topk_group=2)
    assert np.array_equal(host(ids), want_ids)
    if padded:
        q, s, count, h = ep.low_latency_dispatch(x, ids, T, E, format=form)
        spans = [(e * T, int(n)) for e, n in enumerate(host(count))]
    else:
        q, s, _, h = ep.dispatch(x, ids, tw, E, format=form)
        off = host(h.expert_offset)
        spans = [(int(off[e]), int(off[e + 1] - off[e])) for e in range(E)]
    mine = np.zeros(q.numel() // q.shape[-1], dtype=bool)
    for first, n in spans:
        mine[first:first + n] = True

    def product(a, sc, w, ws, act, H, gated):
        y = ep.expert_product(a, sc, w, ws, h, act)
        flat = y.reshape(-1, y.shape[-1])
        av = values(host(a).reshape(len(mine), -1), host(sc).reshape(len(mine), -1))
        av = np.where(mine[:, None], av, 0.0)  # unused rows hold anything
        want, mag = ops.expert_product(av, ops.mxfp4_values(host(w), host(ws)), spans, gated)
        got = flat.view(torch.int16).cpu().numpy().view(np.uint16)
        check(got[mine], want[mine], mag[mine], H, gated)
        return y, flat

    mid, flat = product(q, s, w1, s1, ep.EP_ACT_SWIGLU, H, True)
    q2, sc2 = ep.quantize_rows(flat, form)
    y, _ = product(q2, sc2, w2, s2, ep.EP_ACT_NONE, I, False)
    out = ep.low_latency_combine(y, h, tw) if padded else ep.combine(y, h, tw)
    want = oracle.combine(host(y.reshape(-1, H).view(torch.int16)), host(h.slot), host(tw))
    assert np.array_equal(host(out.view(torch.int16)), want)


def test_routing_trains(gpu):
    """combine's weight gradient, through route_backward, against central
    differences of the loss in 64 bits."""
    ep = gpu
    T, E, K, H = 12, 16, 3, 256
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    logits = torch.randn(T, E, generator=g, device="cuda")
    y = torch.randn(T * K, H, generator=g, device="cuda").bfloat16()
    go = torch.randn(T, H, generator=g, device="cuda").bfloat16()
    ids, w = ep.route(logits, K, scale=2.0)
    h = ep.layout(ids, E)
    _, grad_w = ep.combine_backward(go, y, h, w)
    grad = ep.route_backward(grad_w, logits, ids, scale=2.0).double().cpu().numpy()
    z, idn = logits.double().cpu().numpy(), host(ids)
    yk = y.double().cpu().numpy()[host(h.slot)]  # [T, K, H]
    dots = (yk * go.double().cpu().numpy()[:, None, :]).sum(axis=2)
    mags = np.abs(yk * go.double().cpu().numpy()[:, None, :]).sum(axis=2)

    def loss(zz):
        return (ops.route_weights(zz, idn, ops.SIGMOID, True, 2.0) * dots).sum(axis=1)

    step = 1e-5
    for e in range(E):
        up, down = z.copy(), z.copy()
        up[:, e] += step
        down[:, e] -= step
        d = (loss(up) - loss(down)) / (2 * step)
        # binary32 in both gradients (2^-18 of the terms' magnitudes), and the differences' own curvature and rounding
        tol = 2.0 ** -17 * mags.sum(axis=1) * 2.0 + 1e-8 * (1 + mags.sum(axis=1))
        assert np.all(np.abs(d - grad[:, e]) <= tol)
