"""Routing, quantised rows and the experts' products without a GPU: the
oracle's definitions pinned, and the entry points' refusals."""

import math

import numpy as np
import pytest
import torch

from oracle import operators as ops
from workloads.gen import route_group_limited, route_softmax_topk

FAKE = 0x1000  # never dereferenced: every call below fails validation first


@pytest.fixture(scope="module")
def lib():
    import combine_ep_dispatch_amd as ep

    return ep


# ---- the oracle --------------------------------------------------------------

def test_route_matches_the_workloads_routing():
    """The two routing recipes of the workloads are cases of the rule."""
    z = np.random.default_rng(3).standard_normal((40, 64))
    ids, w = ops.route(z, 8, n_group=8, topk_group=4)
    want_ids, want_w = route_group_limited(z, 8, 4, 8)
    assert np.array_equal(ids, want_ids) and np.allclose(w, want_w, rtol=1e-6)
    ids, w = ops.route(z, 2, score=ops.SOFTMAX)
    want_ids, want_w = route_softmax_topk(z, 2)
    assert np.array_equal(ids, want_ids) and np.allclose(w, want_w, rtol=1e-6)


def test_route_masks_and_ties():
    z = np.zeros((1, 8))
    assert ops.route(z, 3)[0].tolist() == [[0, 1, 2]]  # ties to the lower index
    z[0, :7] = -np.inf
    ids, w = ops.route(z, 3)
    assert ids.tolist() == [[7, -1, -1]] and w.tolist() == [[1.0, 0.0, 0.0]]
    ids, w = ops.route(np.full((1, 8), np.nan), 2, n_group=4, topk_group=2)
    assert ids.tolist() == [[-1, -1]] and not w.any()
    # a group of one choosable expert counts that one alone
    z = np.array([[3.0, -np.inf, 0.0, 0.0]])
    assert ops.route(z, 1, n_group=2, topk_group=1)[0].tolist() == [[2]]  # 0.5 + 0.5 over 0.95
    assert ops.route(np.full((1, 4), -2000.0), 2)[1].tolist() == [[0.5, 0.5]]


@pytest.mark.parametrize("score", [ops.SOFTMAX, ops.SIGMOID])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_backward_against_differences(score, renorm):
    rng = np.random.default_rng(7)
    T, E, K = 5, 12, 4
    z = rng.standard_normal((T, E)) * 2
    z[1, 3] = -np.inf
    ids = np.stack([rng.permutation(E)[:K] for _ in range(T)])
    ids[1, 0], ids[2, 1], ids[3, 2] = 3, -1, ids[3, 0]  # switched off, masked, twice the same
    ids[4, 3] = E + 5
    g = rng.standard_normal((T, K))
    grad, mag = ops.route_backward(g, z, ids, score, renorm, 2.5)
    h = 1e-6
    for t in range(T):
        for e in range(E):
            if np.isneginf(z[t, e]):
                assert grad[t, e] == 0
                continue
            up, down = z.copy(), z.copy()
            up[t, e] += h
            down[t, e] -= h
            d = ((ops.route_weights(up, ids, score, renorm, 2.5) - ops.route_weights(down, ids, score, renorm, 2.5))
                 [t] * g[t]).sum() / (2 * h)
            # central differences: rounding 2^-53 / h per weight of at most 2.5, and curvature h^2
            assert abs(d - grad[t, e]) <= 1e-8 * (1 + np.abs(g[t]).sum() * 2.5)
    assert np.all(mag >= np.abs(grad) * (1 - 1e-12))


def _bits(x):
    return torch.tensor(x, dtype=torch.bfloat16).view(torch.int16).numpy().view(np.uint16)


def test_mxfp4_codes_by_enumeration():
    """Every E2M1 value, midpoint and neighbour of a midpoint, against the
    nearest of the 8 magnitudes with ties to the even code."""
    vals = []
    for a, b in zip(ops.E2M1[:-1], ops.E2M1[1:]):
        mid = (a + b) / 2
        vals += [a, mid * (1 - 2.0 ** -7), mid, mid * (1 + 2.0 ** -7)]
    vals += [6.0, 7.0, 7.75]
    vals += [-v for v in vals]
    for v in vals:
        row = np.zeros((1, 32), dtype=np.float32)
        row[0, 0], row[0, 1] = 4.0, v  # amax in [4, 8): scale 1
        q, s = ops.quantize_mxfp4(_bits(row))
        assert s[0, 0] == 127
        dist = [(abs(min(abs(v), 6.0) - m), i % 2, i) for i, m in enumerate(ops.E2M1)]
        want = min(dist)[2] | (8 if math.copysign(1, v) < 0 else 0)
        assert q[0, 0] == (6 | want << 4), v


def test_mxfp4_scale_edges():
    row = np.zeros((6, 32), dtype=np.float32)
    row[1, 5] = 2.0 ** -126 * 1.5  # floor(log2) - 2 = -128: held at -127
    row[2, 5] = 2.0 ** 127
    row[3, 5] = np.inf
    row[4, 5] = np.nan
    row[5, 5] = -0.0
    q, s = ops.quantize_mxfp4(_bits(row))
    assert s[:, 0].tolist() == [127, 0, 252, 255, 255, 127]
    assert q[1, 2] == 5 << 4 and q[2, 2] == 6 << 4 and q[5, 2] == 8 << 4
    assert not q[3].any() and not q[4].any() and not q[0].any()
    v = ops.mxfp4_values(q, s)
    assert v[1, 5] == 1.5 * 2.0 ** -126 and v[2, 5] == 2.0 ** 127 and np.isnan(v[3]).all()


# ---- refusals ----------------------------------------------------------------

def test_route_rejects_bad_arguments(lib):
    L, bad, uns = lib.LIB, lib.EP_ERR_INVALID_ARG, lib.EP_ERR_UNSUPPORTED
    ok = dict(z=FAKE, dt=0, b=None, T=4, E=16, K=2, ng=4, kg=2, sc=1, rn=1, c=1.0, i=FAKE, w=FAKE)

    def call(**kw):
        a = dict(ok, **kw)
        return L.ep_route(a["z"], a["dt"], a["b"], a["T"], a["E"], a["K"], a["ng"], a["kg"], a["sc"], a["rn"], a["c"],
                          a["i"], a["w"], None)

    assert call(T=-1) == bad and call(E=0) == bad and call(K=0) == bad and call(K=17) == bad
    assert call(E=1025) == uns and call(E=64, K=33) == uns and call(T=1 << 22) == uns
    assert call(dt=2) == bad and call(sc=2) == bad and call(ng=0) == bad and call(ng=3) == bad
    assert call(kg=0) == bad and call(kg=5) == bad and call(E=130, ng=65, kg=1) == uns
    assert call(c=float("nan")) == bad and call(c=float("inf")) == bad
    assert call(z=None) == bad and call(i=None) == bad and call(w=None) == bad
    assert call(z=FAKE + 2) == bad and call(z=FAKE + 1, dt=1) == bad and call(b=FAKE + 2) == bad
    assert call(i=FAKE + 2) == bad and call(w=FAKE + 1) == bad
    assert call(T=0, z=None, i=None, w=None) == lib.EP_OK


def test_route_backward_rejects_bad_arguments(lib):
    L, bad, uns = lib.LIB, lib.EP_ERR_INVALID_ARG, lib.EP_ERR_UNSUPPORTED
    ok = dict(g=FAKE, z=FAKE, dt=0, i=FAKE, T=4, E=16, K=2, sc=1, rn=1, c=1.0, o=FAKE)

    def call(**kw):
        a = dict(ok, **kw)
        return L.ep_route_backward(a["g"], a["z"], a["dt"], a["i"], a["T"], a["E"], a["K"], a["sc"], a["rn"], a["c"],
                                   a["o"], None)

    assert call(T=-1) == bad and call(E=0) == bad and call(K=0) == bad and call(K=17) == bad
    assert call(E=1025) == uns and call(E=64, K=33) == uns
    assert call(dt=-1) == bad and call(sc=-1) == bad and call(c=float("nan")) == bad
    assert call(g=None) == bad and call(z=None) == bad and call(i=None) == bad and call(o=None) == bad
    assert call(g=FAKE + 2) == bad and call(o=FAKE + 2) == bad and call(i=FAKE + 1) == bad
    assert call(T=0, g=None, z=None, i=None, o=None) == lib.EP_OK


def test_rows_reject_bad_arguments(lib):
    mx, fp8 = lib.EP_RECV_MXFP4_G32, lib.EP_RECV_FP8_E4M3_G128
    bad, uns = lib.EP_ERR_INVALID_ARG, lib.EP_ERR_UNSUPPORTED
    for call in (lambda x, r, h, f, q, s: lib.LIB.ep_quantize_rows(x, r, h, f, q, s, None),
                 lambda x, r, h, f, q, s: lib.LIB.ep_dequantize_rows(q, s, r, h, f, x, None)):
        assert call(FAKE, 4, 48, mx, FAKE, FAKE) == bad and call(FAKE, 4, 96, fp8, FAKE, FAKE) == bad
        assert call(FAKE, -1, 128, mx, FAKE, FAKE) == bad and call(FAKE, 4, 0, mx, FAKE, FAKE) == bad
        assert call(FAKE, 4, 128, lib.EP_RECV_BF16, FAKE, FAKE) == bad and call(FAKE, 4, 128, 9, FAKE, FAKE) == bad
        assert call(None, 4, 128, mx, FAKE, FAKE) == bad and call(FAKE, 4, 128, mx, None, FAKE) == bad
        assert call(FAKE, 4, 128, mx, FAKE, None) == bad and call(FAKE + 8, 4, 128, mx, FAKE, FAKE) == bad
        assert call(FAKE, 4, 128, mx, FAKE + 8, FAKE) == bad and call(FAKE, 4, 128, fp8, FAKE, FAKE + 2) == bad
        assert call(FAKE, 1 << 27, 128, mx, FAKE, FAKE) == uns  # rows * H = 2^34
        assert call(FAKE, 1 << 62, 128, mx, FAKE, FAKE) == uns  # no overflow
        assert call(None, 0, 128, mx, None, None) == lib.EP_OK


def test_mxfp4_dispatch_rejects_bad_arguments(lib):
    D, mx, bad = lib.LIB.ep_dispatch, lib.EP_RECV_MXFP4_G32, lib.EP_ERR_INVALID_ARG
    assert D(FAKE, 4, 48, 2, FAKE, None, mx, FAKE, FAKE, None, None) == bad  # H % 32
    assert D(FAKE, 4, 64, 2, FAKE, None, mx, FAKE, None, None, None) == bad  # no scales
    assert D(FAKE, 4, 64, 2, FAKE, None, mx, FAKE + 8, FAKE, None, None) == bad
    assert D(FAKE, 4, 64, 2, None, None, mx, FAKE, FAKE, None, None) == bad
    F = lib.LIB.ep_layout_dispatch
    assert F(FAKE, FAKE, None, 4, 48, 2, 8, 0, mx, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, None, None, 0, None) == bad
    assert F(FAKE, FAKE, None, 4, 64, 2, 8, 0, mx, FAKE, FAKE, FAKE, FAKE, FAKE, None, None, None, 0, None) == bad
    assert D(None, 0, 64, 2, None, None, mx, None, None, None, None) == lib.EP_OK


def test_expert_product_rejects_bad_arguments(lib):
    L, bad, uns = lib.LIB, lib.EP_ERR_INVALID_ARG, lib.EP_ERR_UNSUPPORTED
    ok = dict(a=FAKE, s=FAKE, f=lib.EP_RECV_MXFP4_G32, w=FAKE, ws=FAKE, r=FAKE, R=8, E=4, cap=0, H=256, N=64,
              act=lib.EP_ACT_NONE, y=FAKE)

    def call(**kw):
        a = dict(ok, **kw)
        return L.ep_expert_product(a["a"], a["s"], a["f"], a["w"], a["ws"], a["r"], a["R"], a["E"], a["cap"], a["H"],
                                   a["N"], a["act"], a["y"], None)

    glu = lib.EP_ACT_SWIGLU
    assert call(f=lib.EP_RECV_BF16) == bad and call(f=5) == bad and call(act=2) == bad
    assert call(H=192) == bad and call(H=0) == bad and call(N=0) == bad and call(N=60) == bad
    assert call(N=72, act=glu) == bad and call(R=-1) == bad and call(E=0) == bad and call(cap=-1) == bad
    assert call(cap=3) == bad  # 8 rows are not 4 experts of 3
    assert call(E=1025) == uns and call(H=65536 + 128) == uns and call(N=65536 + 8) == uns
    assert call(R=1 << 31, N=8, H=128) == uns and call(R=1 << 28, H=128, N=8) == uns
    for p in ("a", "s", "w", "ws", "r", "y"):
        assert call(**{p: None}) == bad, p
    for p in ("a", "w", "y"):
        assert call(**{p: FAKE + 8}) == bad, p
    for p in ("s", "ws", "r"):
        assert call(**{p: FAKE + 2}) == bad, p
    assert call(R=0, a=None, s=None, w=None, ws=None, r=None, y=None) == lib.EP_OK


def test_wrappers_refuse_host_tensors_and_wrong_types(lib):
    z = torch.zeros(4, 16)
    with pytest.raises(ValueError, match="GPU device"):
        lib.route(z, 2)
    with pytest.raises(TypeError, match="dtype"):
        lib.route(z.double(), 2)
    with pytest.raises(ValueError, match="top_k"):
        lib.route(z, 0)
    with pytest.raises(ValueError, match="GPU device"):
        lib.route_backward(torch.zeros(4, 2), z, torch.zeros(4, 2, dtype=torch.int32))
    with pytest.raises(ValueError, match="GPU device"):
        lib.quantize_rows(torch.zeros(4, 64, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="format"):
        lib.quantize_rows(torch.zeros(4, 64, dtype=torch.bfloat16), lib.EP_RECV_BF16)
    with pytest.raises(ValueError, match="GPU device"):
        lib.dequantize_rows(torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(4, 2, dtype=torch.uint8))
    h = lib.Handle(None, torch.zeros(3, dtype=torch.int32), None, None, 2)
    with pytest.raises(ValueError, match="GPU device"):
        lib.expert_product(torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(4, 4, dtype=torch.uint8),
                           torch.zeros(2, 16, 64, dtype=torch.uint8), torch.zeros(2, 16, 4, dtype=torch.uint8), h)
    with pytest.raises(ValueError, match="unknown receive format"):
        lib.dispatch(torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(4, 2, dtype=torch.int32), None, 8, format=9)


def test_expert_product_refuses_rows_with_gaps(lib):
    """A copy of them would be made on another stream than the product's."""
    h = lib.Handle(None, torch.zeros(3, dtype=torch.int32), None, None, 2)
    a, s = torch.zeros(4, 128, dtype=torch.uint8), torch.zeros(4, 8, dtype=torch.uint8)
    w, ws = torch.zeros(2, 16, 64, dtype=torch.uint8), torch.zeros(2, 16, 4, dtype=torch.uint8)
    with pytest.raises(ValueError, match="a must be contiguous"):
        lib.expert_product(a[:, :64], s[:, :4].contiguous(), w, ws, h)
    with pytest.raises(ValueError, match="a_scale must be contiguous"):
        lib.expert_product(a[:, :64].contiguous(), s[:, :4], w, ws, h)
    with pytest.raises(ValueError, match="w must be contiguous"):
        lib.expert_product(a[:, :64].contiguous(), s[:, :4].contiguous(), w.transpose(1, 2), ws, h)
