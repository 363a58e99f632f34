"""ep_route and ep_route_backward against the 64-bit oracle.

Ids must be equal.  Weights: the library states 2^-20 relatively.  Gradients:
binary32 terms of a few rounded operations each (exponentials of at most 2
ulp, sums over at most 32 entries as trees or over at most 1024 experts in
per-lane runs and a tree): within 2^-18 of the magnitudes that make up each
element, and half a step of the output type more (bf16: 2^-8 of the value)."""

import numpy as np
import pytest
import torch

from oracle import operators as ops

pytestmark = pytest.mark.gpu


def logits_of(T, E, seed, bf16, spread=1.5):
    z = torch.from_numpy((np.random.default_rng(seed).standard_normal((T, E)) * spread).astype(np.float32))
    return z.to(torch.bfloat16) if bf16 else z


def check_route(ep, z, K, **kw):
    print("case route", tuple(z.shape), z.dtype, K, {k: (v if not isinstance(v, torch.Tensor) else "t") for k, v in kw.items()}, flush=True)
    bias = kw.pop("bias", None)
    ids, w = ep.route(z.cuda(), K, bias=bias.cuda() if bias is not None else None, **kw)
    want_ids, want_w = ops.route(z.double().numpy(), K, bias=None if bias is None else bias.double().numpy(), **kw)
    ids, w = ids.cpu().numpy(), w.double().cpu().numpy()
    assert np.array_equal(ids, want_ids)
    assert np.all(np.abs(w - want_w) <= 2.0 ** -20 * np.abs(want_w) + 2.0 ** -149)
    return ids, w


@pytest.mark.parametrize("T,E,K,groups,kept", [
    (1, 1, 1, 1, 1), (3, 16, 2, 1, 1), (65, 64, 8, 8, 4), (130, 256, 8, 8, 4), (33, 160, 6, 8, 3), (7, 1024, 32, 64, 5),
    (9, 96, 3, 3, 1), (5, 1000, 17, 1, 1), (11, 513, 4, 27, 9), (1025, 256, 8, 8, 4), (6, 40, 32, 2, 2), (64, 8, 8, 4, 2),
    (37, 272, 9, 16, 5), (21, 48, 5, 24, 7), (13, 512, 8, 8, 4), (19, 384, 6, 4, 2)])
@pytest.mark.parametrize("score", [ops.SOFTMAX, ops.SIGMOID])
@pytest.mark.parametrize("bf16", [False, True])
def test_route(gpu, T, E, K, groups, kept, score, bf16):
    z = logits_of(T, E, T * 1000 + E, bf16)
    rng = np.random.default_rng(E)
    for bias in (None, torch.from_numpy((0.1 * rng.standard_normal(E)).astype(np.float32))):
        check_route(gpu, z, K, n_group=groups, topk_group=kept, score=score, bias=bias)
        check_route(gpu, z, K, n_group=groups, topk_group=kept, score=score, bias=bias, renormalize=False, scale=2.5)


@pytest.mark.parametrize("score", [ops.SOFTMAX, ops.SIGMOID])
@pytest.mark.parametrize("E,groups,kept", [(64, 1, 1), (64, 8, 2), (256, 8, 4), (320, 4, 2)])
def test_route_masked_places(gpu, score, E, groups, kept):
    """-inf, NaN and the type's lowest value in places, whole groups, all but
    one expert and all experts of a token; infinities; biases that switch off."""
    z = logits_of(24, E, 5, False)
    n = E // groups
    z[0] = -np.inf
    z[1, 1:] = -np.inf
    z[2, ::2] = float("nan")
    z[3, :n] = -np.inf
    z[4] = float("nan")
    z[5] = torch.finfo(torch.float32).min
    z[6, 3:] = torch.finfo(torch.float32).min
    z[7, 5] = np.inf
    z[8, [4, 9]] = np.inf
    z[9] = -200.0
    z[10] = 100.0
    z[11] = -5000.0
    z[11, 7] = -4999.0
    z[12, :] = 0.0
    z[13, n - 1] = -np.inf
    z[14, 2:] = -np.inf
    check_route(gpu, z, 6, n_group=groups, topk_group=kept, score=score)
    check_route(gpu, z, 6, n_group=groups, topk_group=kept, score=score, renormalize=False)
    bias = torch.zeros(E)
    bias[[1, 8]] = -np.inf
    bias[3] = float("nan")
    bias[5] = -1e30
    check_route(gpu, z[12:], 6, n_group=groups, topk_group=kept, score=score, bias=bias)


@pytest.mark.parametrize("score", [ops.SOFTMAX, ops.SIGMOID])
def test_route_ties_and_near_ties(gpu, score):
    """Equal logits (ties to the lower index), and scores that differ by an
    ulp of binary32, where binary32 arithmetic would lose their order."""
    rng = np.random.default_rng(2)
    E = 256
    z = torch.from_numpy(rng.integers(-2, 3, (64, E)).astype(np.float32))
    check_route(gpu, z, 8, n_group=8, topk_group=4, score=score)
    check_route(gpu, z, 8, n_group=8, topk_group=4, score=score, bias=torch.zeros(E))
    base = rng.standard_normal((64, 1)).astype(np.float32)
    ulps = rng.integers(-3, 4, (64, E)).astype(np.int32)
    z = torch.from_numpy((np.abs(np.broadcast_to(base, (64, E))).copy().view(np.int32) + ulps).view(np.float32))
    check_route(gpu, z, 8, n_group=8, topk_group=4, score=score)
    check_route(gpu, z, 8, n_group=1, topk_group=1, score=score)
    # the bias cancels the scores' differences down to binary32's last bits
    bias = torch.from_numpy((-ops.scores(z[:1].double().numpy(), score)[0]).astype(np.float32))
    check_route(gpu, z, 8, n_group=8, topk_group=4, score=score, bias=bias)


def check_backward(ep, z, ids, g, score, renorm, scale=2.5):
    print("case route_backward", tuple(z.shape), z.dtype, ids.shape[1], score, renorm, flush=True)
    got = ep.route_backward(torch.from_numpy(g).cuda(), z.cuda(), torch.from_numpy(ids).cuda(), score=score, renormalize=renorm,
                            scale=scale)
    assert got.dtype == z.dtype
    want, mag = ops.route_backward(np.where(np.isfinite(g), g, 0), z.double().numpy(), ids, score, renorm, scale)
    got = got.double().cpu().numpy()
    half = 2.0 ** -8 if z.dtype == torch.bfloat16 else 2.0 ** -24
    tol = 2.0 ** -18 * mag
    bad = ~(np.abs(got - want) <= tol + half * (np.abs(want) + tol) + 2.0 ** -126)
    assert not bad.any(), (np.argwhere(bad)[:4], got[bad][:4], want[bad][:4])


@pytest.mark.parametrize("T,E,K", [(1, 1, 1), (3, 16, 2), (65, 256, 8), (7, 1000, 32), (130, 160, 6), (5, 513, 31), (1030, 256, 8), (9, 72, 3)])
@pytest.mark.parametrize("score", [ops.SOFTMAX, ops.SIGMOID])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("bf16", [False, True])
def test_route_backward(gpu, T, E, K, score, renorm, bf16):
    z = logits_of(T, E, 31 * T + E, bf16)
    rng = np.random.default_rng(T)
    ids = np.argsort(rng.random((T, E)), axis=1)[:, :K].astype(np.int32)
    check_backward(gpu, z, ids, rng.standard_normal((T, K)).astype(np.float32), score, renorm)


@pytest.mark.parametrize("score", [ops.SOFTMAX, ops.SIGMOID])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_backward_masked_and_repeated(gpu, score, renorm):
    """Ids out of range and of switched-off experts count for nothing, even
    with NaN in their grad_w; repeated ids add up; extreme logits."""
    rng = np.random.default_rng(9)
    T, E, K = 12, 70, 5
    z = logits_of(T, E, 4, False)
    ids = np.argsort(rng.random((T, E)), axis=1)[:, :K].astype(np.int32)
    g = rng.standard_normal((T, K)).astype(np.float32)
    ids[0] = -1
    g[0] = np.nan
    ids[1, 2], g[1, 2] = E, np.inf
    ids[2, :] = ids[2, 0]
    ids[3, 1], ids[3, 4] = ids[3, 0], ids[3, 2]
    z[4] = -np.inf
    z[5, ids[5, 1]] = float("nan")
    g[5, 1] = np.nan
    z[6, ids[6, 0]] = np.inf
    z[7] = -300.0
    z[8] = 80.0
    ids[9, 0], g[9, 0] = -2 ** 31, np.nan
    ids[10, 3], g[10, 3] = 2 ** 31 - 1, np.nan
    check_backward(gpu, z, ids, g, score, renorm)


def test_route_graph_and_streams(gpu):
    """Captured on a side stream and replayed with new logits between eager
    calls; the backward captured with it."""
    ep = gpu
    T, E, K = 200, 256, 8
    s = torch.cuda.Stream()
    z = logits_of(T, E, 1, False).cuda()
    g = torch.randn(T, K, device="cuda")
    kw = dict(n_group=8, topk_group=4)
    with torch.cuda.stream(s):
        ids, w = ep.route(z, K, **kw)
        d = ep.route_backward(g, z, ids)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        ids, w = ep.route(z, K, **kw)
        d = ep.route_backward(g, z, ids)
    for seed in (2, 3, 4):
        z.copy_(logits_of(T, E, seed, False))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        ids2, w2 = ep.route(z, K, **kw)
        d2 = ep.route_backward(g, z, ids2)
        torch.cuda.synchronize()
        assert torch.equal(ids, ids2) and torch.equal(w, w2) and torch.equal(d, d2)


def test_route_empty_batch(gpu):
    ids, w = gpu.route(torch.zeros(0, 16, device="cuda"), 2)
    assert ids.shape == (0, 2) and w.shape == (0, 2)
    assert gpu.route_backward(w, torch.zeros(0, 16, device="cuda"), ids).shape == (0, 16)


def test_route_refuses_strided_logits(gpu):
    with pytest.raises(ValueError, match="contiguous"):
        gpu.route(torch.zeros(16, 8, device="cuda").t(), 2)
