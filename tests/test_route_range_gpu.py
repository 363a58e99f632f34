"""ep_route and ep_route_backward over the range of their inputs: many
experts, logits far apart, tiny and huge scores.  Ids must be equal to the
oracle's, weights within the stated 2^-20."""

import numpy as np
import pytest
import torch

from oracle import operators as ops
from tests.test_route_gpu import check_route, logits_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("E", [520, 1000, 1024])
def test_softmax_sum_over_many_experts(gpu, E):
    """Twenty-one terms of just under 2^-24 beside a 1: added to it one after
    the other in binary32 they all vanish, while together they are 20 units of
    its last place, enough to change a weight beyond 2^-20 and, with a bias,
    the choice."""
    z = torch.full((3, E), -60.0)
    z[:, 0] = 0.0
    for e in list(range(1, 16)) + [16, 32, 64, 128, 256, 512]:
        z[:, e] = float(np.float32(np.log(2.0 ** -24 * (1 - 2.0 ** -5))))
    ids, w = check_route(gpu, z, 1, score=ops.SOFTMAX, renormalize=False)
    assert ids.tolist() == [[0]] * 3
    bias = torch.full((E,), -5.0)
    bias[0] = 0.0
    bias[E - 1] = 1 - 18 * 2.0 ** -24
    ids, w = check_route(gpu, z, 1, score=ops.SOFTMAX, renormalize=False, bias=bias)
    assert ids.tolist() == [[E - 1]] * 3


@pytest.mark.parametrize("spread", [20.0, 40.0, 80.0])
@pytest.mark.parametrize("score", [ops.SOFTMAX, ops.SIGMOID])
@pytest.mark.parametrize("renorm", [True, False])
def test_weights_of_logits_far_apart(gpu, spread, score, renorm):
    """A difference of logits rounded to binary32 before its exponential would
    be off by up to 2^-18 at 64 and more: four times what is stated.  Smallest
    scores e^-80 / 2^10: above 2^-126."""
    rng = np.random.default_rng(int(spread))
    for T, E, K in [(300, 32, 32), (40, 256, 32), (9, 700, 32)]:
        z = torch.from_numpy((-spread * rng.random((T, E))).astype(np.float32))
        check_route(gpu, z, K, score=score, renormalize=renorm)
        z = torch.from_numpy((spread * (rng.random((T, E)) - 0.5)).astype(np.float32))
        check_route(gpu, z, K, score=score, renormalize=renorm, n_group=4, topk_group=3)


@pytest.mark.parametrize("score", [ops.SOFTMAX, ops.SIGMOID])
@pytest.mark.parametrize("renorm", [True, False])
def test_gradients_of_logits_far_apart(gpu, score, renorm):
    """In units of 2^-24 of the magnitudes that make up an element: an
    exponential 2.4 (1.4 measured, and one), a share of the sum 8 (softmax) or
    12 (renormalised, both sides and three divisions' and conversions'
    roundings), the sum over the K entries 5, products 3, and twice for the
    mean that is taken off: below 40."""
    rng = np.random.default_rng(3)
    for T, E, K in [(2000, 8, 6), (200, 256, 8), (30, 1000, 32)]:
        z = (-85.0 * rng.random((T, E))).astype(np.float32)
        ids = np.argsort(rng.random((T, E)), axis=1)[:, :K].astype(np.int32)
        g = rng.standard_normal((T, K)).astype(np.float32)
        print("case gradients", T, E, K, score, renorm, flush=True)
        got = gpu.route_backward(torch.from_numpy(g).cuda(), torch.from_numpy(z).cuda(), torch.from_numpy(ids).cuda(),
                                 score=score, renormalize=renorm, scale=2.5).double().cpu().numpy()
        want, mag = ops.route_backward(g, z, ids, score, renorm, 2.5)
        bad = ~(np.abs(got - want) <= 40 * 2.0 ** -24 * mag + 2.0 ** -126)
        assert not bad.any(), (int(bad.sum()), got[bad][:4], want[bad][:4])


def test_groups_of_small_scores(gpu):
    """The best groups are those of the largest sums however small these are:
    among scores of e^-60 and e^-30 the latter are chosen."""
    z = torch.full((2, 16), -60.0)
    z[0, 8:] = -30.0
    z[1, 8:] = -59.0
    for score in (ops.SOFTMAX, ops.SIGMOID):
        ids, _ = check_route(gpu, z, 2, n_group=2, topk_group=1, score=score)
        assert ids.tolist() == [[8, 9], [8, 9]]
    ids, _ = check_route(gpu, z, 2, n_group=2, topk_group=1, score=ops.SIGMOID, bias=torch.zeros(16))
    assert ids.tolist() == [[8, 9], [8, 9]]
    rng = np.random.default_rng(4)
    for shift in (-25.0, -60.0, -86.0, -200.0, -700.0):
        for T, E, groups in ((65, 64, 8), (33, 120, 5), (5, 1024, 32)):
            z = torch.from_numpy((shift + 3 * rng.standard_normal((T, E))).astype(np.float32))
            z[1] -= 60 * torch.from_numpy(rng.random(E).astype(np.float32))
            check_route(gpu, z, 4, n_group=groups, topk_group=2, score=ops.SIGMOID)
            z[2, : E // groups] = 0.0  # softmax: the others' scores are small
            check_route(gpu, z, 4, n_group=groups, topk_group=2, score=ops.SOFTMAX)


def test_group_sums_that_are_equal_tie(gpu):
    """s(x) + s(-x) = 1 whatever x: the lower group."""
    x = torch.from_numpy(np.random.default_rng(6).random((200, 1)).astype(np.float32)) * 8
    y = torch.from_numpy(np.random.default_rng(7).random((200, 1)).astype(np.float32)) * 8
    low = torch.full((200, 2), -50.0)
    z = torch.cat([x, -x, low, -y, y, low], 1)
    ids, _ = check_route(gpu, z, 2, n_group=2, topk_group=1)
    assert np.array_equal(np.sort(ids, axis=1), np.broadcast_to([0, 1], (200, 2)))


def test_group_sums_beyond_binary32(gpu):
    """Biases whose sums leave binary32's range, infinite ones among them."""
    z = logits_of(40, 32, 8, False)
    top = float(torch.finfo(torch.float32).max)
    bias = torch.zeros(32)
    for first, second in [((3.0e38, 2.0e38), (3.2e38, 3.1e38)), ((3.0e38, 1.0e38), (top, top)),
                          ((-2.0e38, -3.0e38), (-2.0e38, -2.5e38)), ((3.0e38, 3.0e38), (np.inf, 0.0)),
                          ((np.inf, 1.0), (np.inf, 2.0)), ((np.inf, np.inf), (np.inf, np.inf)), ((1e38, 1e38), (3e38, -1e38))]:
        bias[:8], bias[8:16] = min(first + (0.0,)) - 1.0, min(second + (0.0,)) - 1.0
        bias[[3, 6]], bias[[9, 12]] = torch.tensor(first), torch.tensor(second)
        for score in (ops.SOFTMAX, ops.SIGMOID):
            for kept in (1, 2, 3):
                check_route(gpu, z, 4, n_group=4, topk_group=kept, score=score, bias=bias)
            check_route(gpu, z, 4, n_group=16, topk_group=5, score=score, bias=bias)
            check_route(gpu, z[:, :30].contiguous(), 4, n_group=10, topk_group=2, score=score, bias=bias[:30].contiguous())


@pytest.mark.parametrize("score", [ops.SOFTMAX, ops.SIGMOID])
@pytest.mark.parametrize("renorm", [True, False])
def test_switched_off_by_the_bias(gpu, score, renorm):
    """The bias steers the choice only: the weights are those of the logits
    alone, which is what route_backward differentiates."""
    for E, groups, kept in ((16, 1, 1), (256, 8, 4), (700, 1, 1)):
        z = logits_of(50, E, E, False)
        bias = torch.zeros(E)
        bias[1::3] = -np.inf
        bias[5] = float("nan")
        z[:, 1] = 6.0  # off, and most of softmax's sum
        ids, w = check_route(gpu, z, 4, n_group=groups, topk_group=kept, score=score, bias=bias, renormalize=renorm, scale=2.0)
        want = ops.route_weights(z.double().numpy(), ids, score, renorm, 2.0)
        assert np.all(np.abs(w - want) <= 2.0 ** -20 * want)
        check_route(gpu, z, 4, n_group=groups, topk_group=kept, score=score, bias=torch.full((E,), -np.inf), renormalize=renorm)
