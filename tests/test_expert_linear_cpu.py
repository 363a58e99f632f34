"""The experts' bf16 layers without a GPU: what the C ABI refuses, which
device a call is launched on, and the oracle's gradients against central
differences and brute force."""

import numpy as np
import pytest
import torch

from oracle import operators as ops
from tests.test_devices_cpu import E, H, OnGpu, OnGpu1, T, ep, new  # noqa: F401  (ep is a fixture)

FAKE = 0x1000  # never dereferenced: every call below fails validation first


@pytest.fixture(scope="module")
def lib():
    import combine_ep_dispatch_amd as ep

    return ep


def test_linear_rejects_bad_arguments(lib):
    L, bad, uns = lib.LIB.ep_expert_linear, lib.EP_ERR_INVALID_ARG, lib.EP_ERR_UNSUPPORTED
    none, gated = lib.EP_ACT_NONE, lib.EP_ACT_SWIGLU
    ok = dict(a=FAKE, w=FAKE, b=FAKE, res=FAKE, er=FAKE, R=4, E=2, cap=0, H=64, N=32, act=gated, p=FAKE, y=FAKE)

    def call(**kw):
        k = dict(ok, **kw)
        return L(k["a"], k["w"], k["b"], k["res"], k["er"], k["R"], k["E"], k["cap"], k["H"], k["N"], k["act"], k["p"], k["y"], None)

    assert call(R=-1) == bad and call(E=0) == bad and call(cap=-1) == bad and call(H=0) == bad and call(N=0) == bad
    assert call(H=60) == bad and call(N=24) == bad and call(N=36, act=none, p=None) == bad and call(act=2) == bad
    assert call(act=none) == bad                                  # p belongs to a gated layer
    assert call(E=1025) == uns and call(H=65544) == uns and call(N=65552) == uns
    assert call(R=1 << 31) == uns and call(R=1 << 20, H=1 << 14) == uns and call(R=1 << 20, N=1 << 14) == uns
    assert call(cap=3) == bad                                     # 4 rows are not 2 x 3
    assert call(er=None) == bad and call(er=None, E=1, cap=4) == bad
    for name in ("a", "w", "y"):
        assert call(**{name: None}) == bad
    for name in ("a", "w", "b", "res", "p", "y"):
        assert call(**{name: FAKE + 8}) == bad
    assert call(er=FAKE + 2) == bad
    assert call(R=0, a=None, w=None, y=None) == lib.EP_OK          # no rows: nothing to do


def test_backward_rejects_bad_arguments(lib):
    L, bad, uns = lib.LIB.ep_expert_linear_backward, lib.EP_ERR_INVALID_ARG, lib.EP_ERR_UNSUPPORTED
    ok = dict(g=FAKE, w=FAKE, p=FAKE, er=FAKE, R=4, E=2, cap=0, H=64, N=32, out=FAKE)

    def call(**kw):
        k = dict(ok, **kw)
        return L(k["g"], k["w"], k["p"], k["er"], k["R"], k["E"], k["cap"], k["H"], k["N"], k["out"], None)

    assert call(R=-1) == bad and call(E=0) == bad and call(cap=-1) == bad and call(H=12) == bad and call(N=12) == bad
    assert call(E=1025) == uns and call(H=65544) == uns and call(R=1 << 19, H=1 << 14) == uns  # rows of p are twice as wide
    assert call(cap=3) == bad and call(er=None) == bad and call(er=FAKE + 1) == bad
    for name in ("g", "w", "out"):
        assert call(**{name: None}) == bad and call(**{name: FAKE + 8}) == bad
    assert call(p=FAKE + 4) == bad
    assert call(R=0, g=None, w=None, out=None) == lib.EP_OK


def test_backward_weights_rejects_bad_arguments(lib):
    L, bad, uns = lib.LIB.ep_expert_linear_backward_weights, lib.EP_ERR_INVALID_ARG, lib.EP_ERR_UNSUPPORTED
    ok = dict(g=FAKE, a=FAKE, er=FAKE, R=4, E=2, cap=0, H=64, N=32, t=lib.EP_DTYPE_F32, acc=0, w=FAKE, b=FAKE)

    def call(**kw):
        k = dict(ok, **kw)
        return L(k["g"], k["a"], k["er"], k["R"], k["E"], k["cap"], k["H"], k["N"], k["t"], k["acc"], k["w"], k["b"], None)

    assert call(R=-1) == bad and call(E=0) == bad and call(cap=-1) == bad and call(H=12) == bad and call(N=12) == bad
    assert call(t=2) == bad and call(E=1025) == uns and call(N=65544) == uns and call(R=1 << 20, N=1 << 14) == uns
    assert call(cap=3) == bad and call(er=None) == bad and call(er=FAKE + 2) == bad
    for name in ("g", "a", "w"):
        assert call(**{name: None}) == bad and call(**{name: FAKE + 8}) == bad
    assert call(b=FAKE + 8) == bad
    assert call(R=0, g=None, a=None, acc=1) == lib.EP_OK and call(R=0, w=None) == bad


def calls(ep, cls, odd=None):
    b16, i32 = torch.bfloat16, torch.int32
    n = lambda dtype, *shape: new(cls, dtype, *shape)
    o = lambda dtype, *shape: new(odd or cls, dtype, *shape)
    rows = lambda: n(i32, E + 1)
    yield "ep_expert_linear", lambda: ep.ep_expert_linear(n(b16, T, H), n(b16, E, 16, H), rows(), 0, ep.EP_ACT_SWIGLU, n(b16, T, 8),
                                                          bias=n(b16, E, 16), residual=n(b16, T, 8), p=o(b16, T, 16))
    yield "ep_expert_linear", lambda: ep.ep_expert_linear(n(b16, T, H), n(b16, 1, 16, H), None, 0, ep.EP_ACT_NONE, o(b16, T, 16))
    yield "ep_expert_linear_backward", lambda: ep.ep_expert_linear_backward(n(b16, T, 16), n(b16, E, 16, H), rows(), 0, n(b16, T, 2 * H), p=o(b16, T, 2 * H))
    yield "ep_expert_linear_backward_weights", lambda: ep.ep_expert_linear_backward_weights(n(b16, T, 16), n(b16, T, H), rows(), 0, n(b16, E, 16, H),
                                                                                           o(b16, E, 16), True)


@pytest.mark.parametrize("current", [0, 1])
@pytest.mark.parametrize("cls", [OnGpu, OnGpu1])
def test_launched_on_the_operands_device(ep, cls, current):  # noqa: F811
    ep.current[0] = current
    for name, call in calls(ep.ep, cls):
        ep.calls.clear()
        call()
        assert ep.calls == [(name, cls.index, 100 + cls.index)]
        assert ep.current[0] == current


def test_operands_on_several_devices_are_refused(ep):  # noqa: F811
    for _, call in calls(ep.ep, OnGpu, OnGpu1):
        ep.calls.clear()
        with pytest.raises(ValueError, match="different devices"):
            call()
        assert not ep.calls


def test_oracle_gradients_against_differences():
    """The gated layer and the one behind it: the gradients of p, of the rows,
    of the weights and of the biases against central differences."""
    rng = np.random.default_rng(0)
    spans, H, I, N = [(0, 3), (3, 0), (3, 2)], 4, 3, 5
    a, w1, b1 = rng.standard_normal((6, H)), rng.standard_normal((3, 2 * I, H)), rng.standard_normal((3, 2 * I))
    w2, b2, up = rng.standard_normal((3, N, I)), rng.standard_normal((3, N)), rng.standard_normal((6, N))

    def loss(a, w1, b1, w2, b2):
        mid = ops.expert_linear(a, w1, b1, None, spans, True)["y"][0]
        return np.nansum(up * ops.expert_linear(mid, w2, b2, None, spans, False)["y"][0])

    first = ops.expert_linear(a, w1, b1, None, spans, True)
    gp, _ = ops.expert_linear_backward(up, w2, first["p"][0], spans)
    ga, _ = ops.expert_linear_backward(gp, w1, None, spans)
    g1, g2 = ops.expert_linear_backward_weights(gp, a, spans), ops.expert_linear_backward_weights(up, first["y"][0], spans)
    ga[5] = 0  # a row of no expert
    args = [a, w1, b1, w2, b2]
    for i, grad in enumerate([ga, g1["w"][0], g1["b"][0], g2["w"][0], g2["b"][0]]):
        for at in np.ndindex(args[i].shape):
            step = np.zeros_like(args[i])
            step[at] = 1e-5
            d = (loss(*args[:i], args[i] + step, *args[i + 1:]) - loss(*args[:i], args[i] - step, *args[i + 1:])) / 2e-5
            assert abs(d - grad[at]) < 1e-7 * (1 + abs(d)) + 1e-8, (i, at)


def test_oracle_forward_against_loops():
    rng = np.random.default_rng(1)
    a, w, b, res = rng.standard_normal((5, 3)), rng.standard_normal((2, 4, 3)), rng.standard_normal((2, 4)), rng.standard_normal((5, 2))
    got = ops.expert_linear(a, w, b, res, [(0, 1), (2, 3)], True)
    for r, e in ((0, 0), (2, 1), (3, 1), (4, 1)):
        p = [sum(w[e, n, h] * a[r, h] for h in range(3)) + b[e, n] for n in range(4)]
        assert np.allclose(got["p"][0][r], p)
        assert np.allclose(got["y"][0][r], [p[i] / (1 + np.exp(-p[i])) * p[2 + i] + res[r, i] for i in range(2)])
    assert np.isnan(got["y"][0][1]).all()
