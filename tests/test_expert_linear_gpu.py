"""The experts' bf16 layers and their gradients against the 64-bit oracle.

Two kinds of inputs: small whole numbers, whose sums binary32 holds exactly,
so that the result is the exact sum's rounding bit for bit; and normal ones,
compared within the oracle's bound for binary32 sums plus half a step of the
result's type (2^-8 of the value for BF16, 2^-24 for binary32)."""

import numpy as np
import pytest
import torch

from oracle import operators as ops
from tests.gpu_run import to_dev

pytestmark = pytest.mark.gpu

SENT = 0x7FA5  # a NaN pattern no kernel writes
STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def numbers(rng, shape, whole):
    """bf16 values as float64."""
    if whole:
        return rng.integers(-3, 4, shape).astype(np.float64)
    return torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(torch.bfloat16).double().numpy()


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(torch.bfloat16).cuda() if x is not None else None


def sentinel(*shape):
    return torch.full(shape, SENT, dtype=torch.int16, device="cuda").view(torch.bfloat16)


def check(got, want, bound, whole, name):
    """got: a device tensor; rows whose want is NaN must be as they were."""
    torch.cuda.synchronize()
    mine = ~np.isnan(want)
    if not mine.all():
        bits = got.view(torch.int16).cpu().numpy().view(np.uint16)
        assert np.all(bits[~mine] == SENT), name + ": rows of no expert were written"
    v = got.double().cpu().numpy()
    if whole:
        exact = torch.from_numpy(np.where(mine, want, 0.0)).to(torch.float32).to(got.dtype).double().numpy()
        bad = mine & (v != exact)
    else:
        bad = mine & ~(np.abs(v - want) <= bound + STEP[got.dtype] * (np.abs(want) + bound) + 2.0 ** -133)
    assert not bad.any(), "%s: %d of %d off, first %s: got %r want %r" % (
        name, bad.sum(), mine.sum(), np.argwhere(bad)[0].tolist(), v[bad][0], want[bad][0])


class Rows:
    """The rows of some experts: packed, padded, or (counts an int) one matrix's."""

    def __init__(self, counts, capacity=0, extra=0):
        self.dense = isinstance(counts, int)
        counts = [counts] if self.dense else counts
        self.counts, self.capacity, self.E = counts, capacity, len(counts)
        self.R = self.E * capacity if capacity else sum(counts) + extra
        first = [e * capacity for e in range(self.E)] if capacity else np.concatenate([[0], np.cumsum(counts)]).tolist()
        self.spans = list(zip(first, counts))
        self.dev = None if self.dense else to_dev(np.array(counts if capacity else first, dtype=np.int32))

    def __str__(self):
        return "%s cap %d rows %d" % (self.counts if self.E < 12 else (self.E, max(self.counts)), self.capacity, self.R)


def forward(ep, rows, H, N, gated=False, bias=False, residual=False, save=False, whole=True, seed=0):
    print("case linear", rows, H, N, gated, bias, residual, save, whole, flush=True)
    rng = np.random.default_rng(seed)
    O = N // 2 if gated else N
    a, w = numbers(rng, (rows.R, H), whole), numbers(rng, (rows.E, N, H), whole)
    if not whole:
        w = dev(w / np.sqrt(H)).double().cpu().numpy()
    b = numbers(rng, (rows.E, N), whole) if bias else None
    res = numbers(rng, (rows.R, O), whole) if residual else None
    want = ops.expert_linear(a, w, b, res, rows.spans, gated)
    y, p = sentinel(rows.R, O), sentinel(rows.R, N) if save else None
    ep.ep_expert_linear(dev(a), dev(w), rows.dev, rows.capacity, ep.EP_ACT_SWIGLU if gated else ep.EP_ACT_NONE, y,
                        bias=dev(b), residual=dev(res), p=p)
    check(y, *want["y"], whole and not gated, "y")
    if save:
        check(p, *want["p"], whole, "p")


def backward(ep, rows, H, N, gated=False, whole=True, seed=0):
    print("case rows", rows, H, N, gated, whole, flush=True)
    rng = np.random.default_rng(seed)
    g, w = numbers(rng, (rows.R, N), whole), numbers(rng, (rows.E, N, H), whole)
    if not whole:
        w = dev(w / np.sqrt(N)).double().cpu().numpy()
    p = 3 * numbers(rng, (rows.R, 2 * H), False) if gated else None
    p = dev(p).double().cpu().numpy() if gated else None
    val, bound = ops.expert_linear_backward(g, w, p, rows.spans)
    out = sentinel(rows.R, 2 * H if gated else H)
    ep.ep_expert_linear_backward(dev(g), dev(w), rows.dev, rows.capacity, out, p=dev(p))
    check(out, val, bound, whole and not gated, "grad_a")


def weights(ep, rows, H, N, dtype=torch.bfloat16, bias=True, accumulate=False, whole=True, seed=0):
    print("case weights", rows, H, N, dtype, bias, accumulate, whole, flush=True)
    rng = np.random.default_rng(seed)
    g, a = numbers(rng, (rows.R, N), whole), numbers(rng, (rows.R, H), whole)
    old_w = numbers(rng, (rows.E, N, H), whole) if accumulate else None
    old_b = numbers(rng, (rows.E, N), whole) if accumulate else None
    want = ops.expert_linear_backward_weights(g, a, rows.spans, old_w, old_b)
    grad_w = dev(old_w).to(dtype) if accumulate else torch.full((rows.E, N, H), float("nan"), dtype=dtype, device="cuda")
    grad_b = (dev(old_b).to(dtype) if accumulate else torch.full((rows.E, N), float("nan"), dtype=dtype, device="cuda")) if bias else None
    ep.ep_expert_linear_backward_weights(dev(g), dev(a), rows.dev, rows.capacity, grad_w, grad_b, accumulate)
    check(grad_w, *want["w"], whole, "grad_w")
    if bias:
        check(grad_b, *want["b"], whole, "grad_bias")


COUNTS = [[1], [0, 3, 0], [16, 17, 15, 0, 1, 33], [64, 65, 63], [128, 0, 129, 127, 5], [257, 1, 300], [0, 0, 0, 40], 1, 19, 300]
SIZES = [(8, 16), (40, 64), (136, 208), (256, 512), (648, 272), (1152, 528)]
ids = lambda c: "dense%d" % c if isinstance(c, int) else "-".join(map(str, c))


@pytest.mark.parametrize("whole", [True, False])
@pytest.mark.parametrize("counts", COUNTS, ids=ids)
@pytest.mark.parametrize("H,N", SIZES)
def test_linear(gpu, counts, H, N, whole):
    rows = Rows(counts, extra=0 if isinstance(counts, int) else 3)
    forward(gpu, rows, H, N, whole=whole, seed=H)
    forward(gpu, rows, H, N, gated=True, bias=True, save=True, whole=whole, seed=N)
    forward(gpu, rows, H, N, bias=True, residual=True, whole=whole, seed=1)
    forward(gpu, rows, H, N, gated=True, residual=True, whole=whole, seed=2)


@pytest.mark.parametrize("whole", [True, False])
@pytest.mark.parametrize("counts", COUNTS, ids=ids)
@pytest.mark.parametrize("H,N", [(16, 8)] + SIZES[1:])
def test_linear_backward(gpu, counts, H, N, whole):
    rows = Rows(counts, extra=0 if isinstance(counts, int) else 3)
    backward(gpu, rows, H, N, whole=whole, seed=H)
    backward(gpu, rows, H, N, gated=True, whole=whole, seed=N)


@pytest.mark.parametrize("whole", [True, False])
@pytest.mark.parametrize("counts", COUNTS, ids=ids)
@pytest.mark.parametrize("H,N", [(8, 8)] + SIZES[1:])
def test_linear_backward_weights(gpu, counts, H, N, whole):
    rows = Rows(counts, extra=0 if isinstance(counts, int) else 3)
    weights(gpu, rows, H, N, whole=whole, seed=H)
    weights(gpu, rows, H, N, dtype=torch.float32, bias=False, whole=whole, seed=N)
    weights(gpu, rows, H, N, dtype=torch.float32, accumulate=True, whole=whole, seed=1)
    weights(gpu, rows, H, N, accumulate=True, whole=whole, seed=2)


@pytest.mark.parametrize("whole", [True, False])
@pytest.mark.parametrize("H,N", [(8, 8), (24, 1000), (896, 24), (2048, 136), (56, 8)])
def test_narrow(gpu, H, N, whole):
    """Channel counts that are multiples of 8 only."""
    for counts in ([3, 0, 70, 1], 5):
        forward(gpu, Rows(counts), H, N, bias=True, whole=whole)
        backward(gpu, Rows(counts), H, N, whole=whole)
        weights(gpu, Rows(counts), H, N, whole=whole)


@pytest.mark.parametrize("whole", [True, False])
@pytest.mark.parametrize("counts,capacity", [([0, 5, 1, 9], 9), ([128, 3, 0], 128), ([40, 33], 47), ([1, 1, 1, 0, 1], 1), ([300, 2, 0, 299], 300)])
def test_padded(gpu, counts, capacity, whole):
    rows = Rows(counts, capacity)
    for H, N in ((768, 160), (200, 544)):
        forward(gpu, rows, H, N, gated=True, bias=True, residual=True, save=True, whole=whole)
        forward(gpu, rows, H, N, whole=whole)
        backward(gpu, rows, H, N, whole=whole)
        backward(gpu, rows, H, N, gated=True, whole=whole)
        weights(gpu, rows, H, N, whole=whole)


def test_many_experts(gpu):
    rng = np.random.default_rng(1)
    few = Rows(rng.integers(0, 3, 1024).tolist())
    forward(gpu, few, 64, 32)
    backward(gpu, few, 64, 32)
    weights(gpu, few, 64, 32)
    some = Rows((rng.integers(0, 40, 100) * (rng.random(100) < 0.5)).astype(int).tolist())
    forward(gpu, some, 256, 96, gated=True, whole=False)
    backward(gpu, some, 256, 96, gated=True, whole=False)
    weights(gpu, some, 256, 96, whole=False)


@pytest.mark.parametrize("counts", [[515, 260, 1023], [1, 2000], 1300], ids=ids)
@pytest.mark.parametrize("H,N", [(1024, 592), (264, 1552), (4104, 32)])
def test_large_rows(gpu, counts, H, N):
    """Enough rows per expert for the largest tiles, with ragged ends."""
    rows = Rows(counts)
    forward(gpu, rows, H, N, gated=True, bias=True, residual=True, save=True)
    forward(gpu, rows, H, N, bias=True, residual=True)
    backward(gpu, rows, H, N)
    backward(gpu, rows, H, N, gated=True)
    weights(gpu, rows, H, N)
    weights(gpu, rows, H, N, dtype=torch.float32, accumulate=True)


@pytest.mark.parametrize("H", [64, 128, 192, 328, 648])
@pytest.mark.parametrize("experts,rows,N", [(45, 5, 1536), (24, 50, 1312), (12, 130, 2944), (7, 300, 2560)])
def test_stages(gpu, experts, rows, N, H):
    """Sums of one to many stages, each tile, several tiles in turn on a workgroup."""
    rng = np.random.default_rng(H)
    r = Rows(rng.integers(0, 2 * rows + 1, experts).tolist())
    forward(gpu, r, H, N, gated=N % 512 == 0, bias=True, seed=H)
    forward(gpu, r, N, H, seed=H)
    backward(gpu, r, N, H, seed=H)
    backward(gpu, r, H, N, gated=True, seed=H)
    weights(gpu, r, H, N, seed=H)


BAD = [([-5, 100, 50, 100000, 7], 0, [(0, 100), (100, 0), (50, 350), (400, 0)]),
       ([2 ** 31 - 1, -2 ** 31, 3, 3, 3], 0, [(400, 0), (0, 3), (3, 0), (3, 0)]),
       ([999, -3, 100, 2 ** 31 - 1], 100, [(0, 100), (100, 0), (200, 100), (300, 100)])]


@pytest.mark.parametrize("er,cap,spans", BAD)
def test_bad_spans_are_clamped(gpu, er, cap, spans):
    """Offsets and counts outside the buffer."""
    ep = gpu
    rng = np.random.default_rng(0)
    H, N, R = 136, 48, 400
    a, w, g = numbers(rng, (R, H), True), numbers(rng, (4, N, H), True), numbers(rng, (R, N), True)
    er = to_dev(np.array(er, dtype=np.int32))
    print("case spans", er.tolist(), cap, flush=True)
    shared = slice(50, 100) if spans[2] == (50, 350) else slice(0, 0)  # rows of two experts: one of the two writes last

    def cut(x):
        return np.delete(x, np.arange(R)[shared], 0)

    y, grad_a, grad_w = sentinel(R, N), sentinel(R, H), torch.empty(4, N, H, device="cuda")
    ep.ep_expert_linear(dev(a), dev(w), er, cap, ep.EP_ACT_NONE, y)
    ep.ep_expert_linear_backward(dev(g), dev(w), er, cap, grad_a)
    ep.ep_expert_linear_backward_weights(dev(g), dev(a), er, cap, grad_w)
    keep = torch.from_numpy(cut(np.arange(R))).cuda()
    check(y[keep], cut(ops.expert_linear(a, w, None, None, spans, False)["y"][0]), 0, True, "y")
    check(grad_a[keep], cut(ops.expert_linear_backward(g, w, None, spans)[0]), 0, True, "grad_a")
    check(grad_w, *ops.expert_linear_backward_weights(g, a, spans)["w"], True, "grad_w")


@pytest.mark.parametrize("H,N", [(72, 48), (640, 336)])
def test_nan_and_infinity_stay_where_they_are(gpu, H, N):
    """In a row, a channel or another expert's rows; weights of channels past
    the end and rows past an expert's end never count."""
    ep = gpu
    rng = np.random.default_rng(H)
    rows = Rows([70, 0, 3, 40], extra=2)
    a, w, g = numbers(rng, (rows.R, H), True), numbers(rng, (4, N, H), True), numbers(rng, (rows.R, N), True)
    a[2, H - 3], a[71, 5], a[113] = np.nan, np.inf, np.nan  # experts 0 and 2, and a row of no expert
    g[2, 1], g[113], g[72, N - 1] = np.nan, np.inf, np.inf
    w[1] = np.nan  # an expert without rows
    w[3, 7, 2] = np.nan
    print("case nan", H, N, flush=True)

    def same(got, want):
        torch.cuda.synchronize()
        got = got.double().cpu().numpy()
        mine = ~np.isnan(want)
        assert np.array_equal(np.isnan(got), np.isnan(want))
        with np.errstate(invalid="ignore"):
            exact = torch.from_numpy(want).to(torch.float32).to(torch.bfloat16).double().numpy()
        assert np.array_equal(got[mine], exact[mine])

    y, grad_a, grad_w = sentinel(rows.R, N), sentinel(rows.R, H), torch.empty(4, N, H, dtype=torch.bfloat16, device="cuda")
    ep.ep_expert_linear(dev(a), dev(w), rows.dev, 0, ep.EP_ACT_NONE, y)
    ep.ep_expert_linear_backward(dev(g), dev(w), rows.dev, 0, grad_a)
    ep.ep_expert_linear_backward_weights(dev(g), dev(a), rows.dev, 0, grad_w)
    with np.errstate(invalid="ignore"):
        same(y[:113], ops.expert_linear(a, w, None, None, rows.spans, False)["y"][0][:113])
        same(grad_a[:113], ops.expert_linear_backward(g, w, None, rows.spans)[0][:113])
        same(grad_w, ops.expert_linear_backward_weights(g, a, rows.spans)["w"][0])


def test_activation_far_out(gpu):
    """Pre-activations from -90 to 90 and around the slope's zero: both sides
    of the gate, within their bounds."""
    ep = gpu
    H, R = 256, 180
    grid = np.concatenate([np.linspace(-90, 90, H - 64), np.linspace(-1.35, -1.2, 64)])
    p = dev(np.tile(np.concatenate([grid, np.linspace(-2, 2, H)]), (R, 1))).double().cpu().numpy()
    rng = np.random.default_rng(0)
    g, w = numbers(rng, (R, 64), False), numbers(rng, (1, 64, H), False)
    val, bound = ops.expert_linear_backward(g, w, p, [(0, R)])
    out = sentinel(R, 2 * H)
    ep.ep_expert_linear_backward(dev(g), dev(w), None, 0, out, p=dev(p))
    check(out, val, bound, False, "grad_p")
    # forward: one input channel carries the pre-activation
    a, w = np.zeros((R, 8)), np.zeros((1, 2 * H, 8))
    a[:, 0], w[0, :, 0] = 1, p[0]
    want = ops.expert_linear(a, w, None, None, [(0, R)], True)
    y = sentinel(R, H)
    ep.ep_expert_linear(dev(a), dev(w), None, 0, ep.EP_ACT_SWIGLU, y)
    check(y, *want["y"], False, "y")


def test_in_place(gpu):
    """y over its residual, the gradient of p over p."""
    ep = gpu
    rng = np.random.default_rng(4)
    for R, H, N in ((5, 264, 144), (700, 136, 528)):
        a, w, res = numbers(rng, (R, H), True), numbers(rng, (1, N, H), True), numbers(rng, (R, N), True)
        y = dev(res)
        ep.ep_expert_linear(dev(a), dev(w), None, 0, ep.EP_ACT_NONE, y, residual=y)
        check(y, *ops.expert_linear(a, w, None, res, [(0, R)], False)["y"], True, "y")
        g, p = numbers(rng, (R, N), False), numbers(rng, (R, 2 * H), False)
        out = dev(p)
        ep.ep_expert_linear_backward(dev(g), dev(w), None, 0, out, p=out)
        check(out, *ops.expert_linear_backward(g, w, p, [(0, R)]), False, "grad_p")


@pytest.mark.parametrize("E,H,N,counts", [(8, 1024, 512, [3, 0, 200, 17, 64, 1, 130, 40]), (2, 256, 128, [1, 2])])
def test_repeats_bitwise_on_streams_and_in_graphs(gpu, E, H, N, counts):
    """The same bits on every run: on two side streams at once, and captured
    and replayed between eager calls."""
    ep = gpu
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    off = torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32, device="cuda")
    R = sum(counts)
    new = lambda *shape: torch.randn(*shape, generator=g, device="cuda").bfloat16()
    a, w, b, go, res = new(R, H), new(E, N, H), new(E, N), new(R, N), new(R, N // 2)
    h = ep.Handle(None, off, None, None, E)

    def step():
        y, p = ep.expert_linear(a, w, h, b, ep.EP_ACT_SWIGLU, res, save=True)
        return (y, p, ep.expert_linear_backward(go, w, h), ep.expert_linear_backward(p, w, h, p=torch.cat([a, a], 1)),
                *ep.expert_linear_backward_weights(go, a, h, torch.float32, bias=True))

    want = step()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = []
    for _ in range(4):
        for st in streams:
            with torch.cuda.stream(st):
                outs.append(step())
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for o in outs for x, y in zip(o, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=streams[0]):
        y = step()
    for k in range(3):
        a.copy_(a.roll(1, 0))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        eager = step()
        torch.cuda.synchronize()
        assert all(torch.equal(x, z) for x, z in zip(y, eager))


def test_empty(gpu):
    ep = gpu
    h = ep.Handle(None, torch.zeros(3, dtype=torch.int32, device="cuda"), None, None, 2)
    z = lambda *n: torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    assert ep.expert_linear(z(0, 64), z(2, 16, 64), h).shape == (0, 16)
    assert ep.expert_linear_backward(z(0, 16), z(2, 16, 64), h, p=z(0, 128)).shape == (0, 128)
    for rows in (0, 5):  # no rows at all, and rows of no expert
        for dtype in (torch.bfloat16, torch.float32):
            gw, gb = torch.full((2, 16, 64), 3.0, dtype=dtype, device="cuda"), torch.full((2, 16), 3.0, dtype=dtype, device="cuda")
            ep.ep_expert_linear_backward_weights(z(rows, 16), z(rows, 64), h.expert_offset, 0, gw, gb, True)
            assert bool((gw == 3).all()) and bool((gb == 3).all())
            ep.ep_expert_linear_backward_weights(z(rows, 16), z(rows, 64), h.expert_offset, 0, gw, gb)
            assert not bool(gw.any()) and not bool(gb.any())


def test_refuses_mismatched_operands(gpu):
    ep = gpu
    z = lambda *n: torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    h = ep.Handle(None, torch.zeros(3, dtype=torch.int32, device="cuda"), None, None, 2)
    bad = [lambda: ep.expert_linear(z(4, 56), z(2, 16, 64), h), lambda: ep.expert_linear(z(4, 64), z(2, 20, 64), h),
           lambda: ep.expert_linear(z(4, 64), z(3, 16, 64), h), lambda: ep.expert_linear(z(4, 60), z(2, 16, 60), h),
           lambda: ep.expert_linear(z(4, 64), z(2, 24, 64), h, activation=ep.EP_ACT_SWIGLU),
           lambda: ep.expert_linear(z(4, 64), z(2, 16, 64), h, save=True), lambda: ep.expert_linear(z(4, 64), z(2, 16, 64), None),
           lambda: ep.expert_linear(z(4, 64), z(2, 16, 64), h, bias=z(16)), lambda: ep.expert_linear(z(4, 64), z(2, 16, 64), h, residual=z(4, 8)),
           lambda: ep.expert_linear(z(64, 4).t(), z(2, 16, 64), h), lambda: ep.expert_linear(z(4, 64), z(2, 64, 16).transpose(1, 2), h),
           lambda: ep.expert_linear(z(4, 64), z(2, 16, 64), h, activation=7),
           lambda: ep.expert_linear_backward(z(4, 24), z(2, 16, 64), h), lambda: ep.expert_linear_backward(z(4, 16), z(2, 16, 64), h, p=z(4, 64)),
           lambda: ep.expert_linear_backward_weights(z(4, 16), z(5, 64), h), lambda: ep.expert_linear_backward_weights(z(4, 16), z(4, 60), h),
           lambda: ep.ep_expert_linear(z(4, 64), z(2, 16, 64), torch.zeros(2, dtype=torch.int32, device="cuda"), 3, ep.EP_ACT_NONE, z(4, 16))]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    for call in (lambda: ep.expert_linear(z(4, 64).float(), z(2, 16, 64), h), lambda: ep.expert_linear(z(4, 64), z(2, 16, 64).half(), h),
                 lambda: ep.expert_linear(z(4, 64), z(2, 16, 64), h, bias=z(2, 16).float()),
                 lambda: ep.expert_linear_backward_weights(z(4, 16), z(4, 64), h, dtype=torch.float16)):
        with pytest.raises(TypeError):
            call()


def test_rows_and_weights_beyond_32_bits(gpu):
    """Rows, weights and gradients more than 2^32 bytes into their buffers."""
    ep = gpu
    rng = np.random.default_rng(3)
    H, N, E, R, n = 32768, 72, 1000, 70000, 37
    assert E * N * H * 2 > 2 ** 32 and R * H * 2 > 2 ** 32
    a, w, g = numbers(rng, (n, H), True), numbers(rng, (N, H), True), numbers(rng, (n, N), True)
    da, dw = torch.zeros(R, H, dtype=torch.bfloat16, device="cuda"), torch.zeros(E, N, H, dtype=torch.bfloat16, device="cuda")
    dg = torch.zeros(R, N, dtype=torch.bfloat16, device="cuda")
    da[R - n:], dw[E - 1], dg[R - n:] = dev(a), dev(w), dev(g)
    off = torch.full((E + 1,), R - n, dtype=torch.int32, device="cuda")
    off[E] = R
    print("case beyond 32 bits", flush=True)
    y, grad_a = sentinel(R, N), sentinel(R, H)
    ep.ep_expert_linear(da, dw, off, 0, ep.EP_ACT_NONE, y)
    ep.ep_expert_linear_backward(dg, dw, off, 0, grad_a)
    spans = [(0, n)]
    check(y[R - n:], *ops.expert_linear(a, w[None], None, None, spans, False)["y"], True, "y")
    check(grad_a[R - n:], *ops.expert_linear_backward(g, w[None], None, spans), True, "grad_a")
    assert bool((y[:R - n].view(torch.int16) == SENT).all()) and bool((grad_a[:R - n].view(torch.int16) == SENT).all())
    grad_w = torch.full((E, N, H), 5.0, dtype=torch.bfloat16, device="cuda")
    ep.ep_expert_linear_backward_weights(dg, da, off, 0, grad_w)
    check(grad_w[E - 1:], *ops.expert_linear_backward_weights(g, a, spans)["w"], True, "grad_w")
    assert not bool(grad_w[:E - 1].any())


def test_one_expert_with_rows_over_4_gib(gpu):
    """A single expert's rows span more than 2^32 bytes: its last rows count."""
    ep = gpu
    rng = np.random.default_rng(7)
    H, N, R, n = 65536, 16, 33000, 40
    da, dg = torch.zeros(R, H, dtype=torch.bfloat16, device="cuda"), torch.zeros(R, N, dtype=torch.bfloat16, device="cuda")
    a, g, w = numbers(rng, (n, H), True), numbers(rng, (n, N), True), numbers(rng, (1, N, H), True)
    da[R - n:], dg[R - n:] = dev(a), dev(g)
    print("case 4 GiB of one expert", flush=True)
    grad_w = torch.empty(1, N, H, dtype=torch.bfloat16, device="cuda")
    ep.ep_expert_linear_backward_weights(dg, da, None, 0, grad_w)
    check(grad_w, *ops.expert_linear_backward_weights(g, a, [(0, n)])["w"], True, "grad_w")
    y = ep.expert_linear(da, dev(w), None)
    check(y[R - n:], *ops.expert_linear(a, w, None, None, [(0, n)], False)["y"], True, "y")
    assert not bool(y[:R - n].any())
