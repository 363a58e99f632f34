"""The sums of the experts' bf16 layers are binary32, in every tile and every
place of a sum: terms 2^-23 below the sum they meet, large terms that cancel,
and subnormal factors, products and results.

Every input here is such that each partial sum, in any order, is a multiple
of one unit below 2^24 of it: binary32 holds all of them, so the result is the
exact sum, bit for bit.  A matrix unit that drops low bits of the terms it adds
together, or flushes subnormals, gives another one."""

import numpy as np
import pytest
import torch

from oracle import operators as ops
from tests.test_expert_linear_gpu import Rows, check, dev, sentinel
from tests.test_expert_linear_tiles_gpu import TILES, rows_of

pytestmark = pytest.mark.gpu


def cancelling(rng, R, N, C):
    """x [R, C], w [N, C] of whole numbers up to 255, whose products cancel but
    for one a row of w: sums of at most 255, magnitudes that add up to less than
    2^24."""
    most = min(255, int((2 ** 24 / C) ** 0.5) - 1)
    x, w = np.zeros((R, C)), np.zeros((N, C))
    at = rng.permutation(C)
    one, other = at[: C // 2], at[C // 2:]
    x[:, one] = rng.integers(-most, most + 1, (R, C // 2))
    x[:, other] = x[:, one]
    w[:, one] = rng.integers(-most + 1, most, (N, C // 2))
    w[:, other] = -w[:, one]
    w[np.arange(N), other[rng.integers(0, C // 2, N)]] += rng.choice([-1, 1], N)
    assert (np.abs(x).max(0) * np.abs(w).max(0)).sum() < 2 ** 24
    return x, w


@pytest.mark.parametrize("C", [248, 2056])
@pytest.mark.parametrize("tile", TILES)
def test_large_terms_cancel_exactly(gpu, tile, C):
    ep = gpu
    rows, O = TILES[tile]
    r = rows_of(rows)
    rng = np.random.default_rng(C)
    print("case cancel", tile, C, flush=True)
    x, one = cancelling(rng, r.R, O, C)
    want = ops.expert_linear(x, np.broadcast_to(one, (r.E, O, C)), None, None, r.spans, False)["y"]
    assert np.nanmax(np.abs(want[0])) <= 255
    w, y = dev(one).expand(r.E, O, C), sentinel(r.R, O)
    x = dev(x)
    ep.ep_expert_linear(x, w.contiguous(), r.dev, r.capacity, ep.EP_ACT_NONE, y)
    check(y, *want, True, "y")
    # the rows of a gated layer before its activation
    wide = sentinel(r.R, O // 16 * 16)
    ep.ep_expert_linear(x, w[:, : O // 16 * 16].contiguous(), r.dev, r.capacity, ep.EP_ACT_SWIGLU, sentinel(r.R, O // 16 * 8), p=wide)
    check(wide, want[0][:, : O // 16 * 16], want[1][:, : O // 16 * 16], True, "p")
    grad_a = sentinel(r.R, O)
    ep.ep_expert_linear_backward(x, w.transpose(1, 2).contiguous(), r.dev, r.capacity, grad_a)
    check(grad_a, *want, True, "grad_a")


WEIGHTS = [([1000, 0, 1, 450, 900], 1800, 2304), ([40] * 70, 600, 704), (2056, 304, 200), ([64, 0, 70], 136, 520), (257, 8, 16), (32768, 264, 520)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("counts,H,N", WEIGHTS, ids=lambda c: str(c) if isinstance(c, int) else "x".join(map(str, c[:3])))
def test_large_terms_cancel_exactly_in_weights(gpu, counts, H, N, dtype):
    ep = gpu
    r = Rows(counts)
    rng = np.random.default_rng(H)
    print("case cancel weights", r, H, N, dtype, flush=True)
    g, a = np.zeros((r.R, N)), np.zeros((r.R, H))
    for first, n in r.spans:
        if n > 1:
            at = slice(first, first + n // 2 * 2)
            x, w = cancelling(rng, N, H, n // 2 * 2)
            g[at], a[at] = x.T, w.T
    want = ops.expert_linear_backward_weights(g, a, r.spans)
    grad_w = torch.full((r.E, N, H), float("nan"), dtype=dtype, device="cuda")
    ep.ep_expert_linear_backward_weights(dev(g), dev(a), r.dev, 0, grad_w)
    check(grad_w, *want["w"], True, "grad_w")
    # onto an old gradient
    old = rng.integers(-255, 256, grad_w.shape).astype(np.float64)
    grad_w = dev(old).to(dtype)
    ep.ep_expert_linear_backward_weights(dev(g), dev(a), r.dev, 0, grad_w, accumulate=True)
    check(grad_w, want["w"][0] + old, want["w"][1], True, "grad_w, accumulated")


def test_terms_2_23_below_the_sum(gpu):
    """1 and 2^-23 in every two places of a sum, with -1 in a third, or as the
    bias: 2^-23 is left."""
    ep = gpu
    C, rng = 128, np.random.default_rng(0)
    i, j = (v.ravel() for v in np.meshgrid(np.arange(C), np.arange(C), indexing="ij"))
    i, j = i[i != j], j[i != j]
    k = (np.maximum(i, j) + 1 + rng.integers(0, C - 2, len(i))) % C
    k = np.where((k == i) | (k == j), (k + 1) % C, k)
    k = np.where((k == i) | (k == j), (k + 1) % C, k)
    R, at = len(i), np.arange(len(i))
    w = np.ones((C, C))
    w[np.arange(C), np.arange(C)] = 2.0 ** -11  # channel n: at place n
    for third in (True, False):
        print("case low term", third, flush=True)
        x = np.zeros((R, C))
        x[at, i], x[at, j] = 1, 2.0 ** -12
        bias = None
        if third:
            x[at, k] = -1
        else:
            bias = dev(-np.ones((1, C)))
        picked = (torch.from_numpy(at).cuda(), torch.from_numpy(j).cuda())
        for every in (1, 25, 150, 1000):  # (of the rows: large tiles, small ones, groups of waves, few rows)
            part, place = dev(x)[::every].contiguous(), picked[1][::every]
            row = torch.arange(len(place)).cuda()
            y = ep.expert_linear(part, dev(w)[None], None, bias=bias)
            assert bool((y[row, place].double() == 2.0 ** -23).all()), "y"
            if third:
                grad = ep.expert_linear_backward(part, dev(w.T)[None], None)
                assert bool((grad[row, place].double() == 2.0 ** -23).all()), "grad_a"
        if third:  # summed over C rows: column r of the result holds the terms of row r above
            grad_w = ep.expert_linear_backward_weights(dev(w.T), dev(x.T), None, dtype=torch.float32)[0]
            assert bool((grad_w[picked[1], picked[0]] == 2.0 ** -23).all()), "grad_w"


@pytest.mark.parametrize("ax,wx", [(-133, 0), (0, -133), (-80, -53), (-126, -7)])
@pytest.mark.parametrize("rows", [13, 100, 600, 1300])
def test_subnormals(gpu, rows, ax, wx):
    """Subnormal factors, products and results: whole numbers times 2^-133,
    BF16's lowest value."""
    ep = gpu
    rng = np.random.default_rng(rows)
    C, O = 136, 1000
    x, w = rng.integers(-3, 4, (rows, C)) * 2.0 ** ax, rng.integers(-3, 4, (O, C)) * 2.0 ** wx
    want = x @ w.T
    r = Rows(rows)
    print("case subnormal", rows, ax, wx, flush=True)
    y, grad_a = sentinel(rows, O), sentinel(rows, O)
    ep.ep_expert_linear(dev(x), dev(w)[None], None, 0, ep.EP_ACT_NONE, y)
    ep.ep_expert_linear_backward(dev(x), dev(np.ascontiguousarray(w.T))[None], None, 0, grad_a)

    def same(got, want, name):
        exact = torch.from_numpy(want).to(torch.float32).to(got.dtype).double().numpy()
        v = got.double().cpu().numpy()
        assert np.array_equal(v, exact), "%s: %d off" % (name, (v != exact).sum())

    same(y, want, "y")
    same(grad_a, want, "grad_a")
    for dtype in (torch.bfloat16, torch.float32):
        grad_w = torch.empty(1, rows // 8 * 8, O, dtype=dtype, device="cuda")
        ep.ep_expert_linear_backward_weights(dev(np.ascontiguousarray(x.T)[:, : rows // 8 * 8]), dev(np.ascontiguousarray(w.T)), None, 0, grad_w)
        same(grad_w[0], want[: rows // 8 * 8], "grad_w")


def test_gates_whose_sigmoid_is_below_binary32(gpu):
    """Gates from -170 to -85, whose sigmoid is down to 2^-245, with factors
    around it that bring the results back: within the oracle's bound."""
    ep = gpu
    H, R = 176, 180
    gate, up = np.linspace(-170, -85, H), 2.0 ** np.linspace(100, 126, H)[::-1]
    p = dev(np.tile(np.concatenate([gate, up]), (R, 1))).double().cpu().numpy()
    rng = np.random.default_rng(0)
    g = dev(rng.standard_normal((R, 64)) * 2.0 ** 60).double().cpu().numpy()
    w = dev(rng.standard_normal((1, 64, H)) * 2.0 ** np.linspace(60, 10, H)).double().cpu().numpy()
    val, bound = ops.expert_linear_backward(g, w, p, [(0, R)])
    assert np.abs(val[:, :H]).min() > 2.0 ** -120 and np.abs(val).max() < 2.0 ** 127
    out = sentinel(R, 2 * H)
    ep.ep_expert_linear_backward(dev(g), dev(w), None, 0, out, p=dev(p))
    check(out, val, bound, False, "grad_p")
    # forward: one input channel carries the pre-activation
    a, w = np.zeros((R, 8)), np.zeros((1, 2 * H, 8))
    a[:, 0], w[0, :, 0] = 1, p[0]
    want = ops.expert_linear(a, w, None, None, [(0, R)], True)["y"]
    assert np.abs(want[0]).min() > 2.0 ** -126
    y = sentinel(R, H)
    ep.ep_expert_linear(dev(a), dev(w), None, 0, ep.EP_ACT_SWIGLU, y)
    check(y, *want, False, "y")


def test_a_long_sum_is_the_same_in_both_types(gpu):
    """32768 rows of one matrix: the same bits on every run, BF16 the rounding
    of the binary32 sums, and both within their bound."""
    ep = gpu
    R, H, N = 32768, 264, 520
    rng = np.random.default_rng(2)
    g, a = dev(rng.standard_normal((R, N))), dev(rng.standard_normal((R, H)))
    print("case long sum", flush=True)
    wide = ep.expert_linear_backward_weights(g, a, None, torch.float32, bias=True)
    narrow = ep.expert_linear_backward_weights(g, a, None, bias=True)
    for _ in range(3):
        again = ep.expert_linear_backward_weights(g, a, None, torch.float32, bias=True)
        assert all(torch.equal(x, y) for x, y in zip(wide, again))
    assert all(torch.equal(x.bfloat16(), y) for x, y in zip(wide, narrow))
    want = ops.expert_linear_backward_weights(g.double().cpu().numpy(), a.double().cpu().numpy(), [(0, R)])
    for got in (wide, narrow):
        check(got[0], *want["w"], False, "grad_w")
        check(got[1], *want["b"], False, "grad_bias")
