"""ep_expert_product against the 64-bit oracle.

Bound per element: with p the exact sum and m = sum_h |w a|, the binary32
sum of H exact products is within H * 2^-23 * m of p (every addition off by
at most one unit of the last place of a partial sum, rounded or truncated),
FP8 rows add two rounded operations per 128 channels; the activation carries
that through its slopes (|silu'| <= 1.1) and adds 2^-19 of the value (one
exponential, a division and a product); rounding to BF16 is half a step,
2^-8 of the value at most."""

import numpy as np
import pytest
import torch

import oracle
from oracle import operators as ops
from tests.gpu_run import SENT_BF16, to_dev

pytestmark = pytest.mark.gpu


def bf16_bits(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16)


def rows_of(rng, rows, H, fmt):
    """-> codes, scales (host), values."""
    x = bf16_bits(rng.standard_normal((rows, H)) * np.exp(0.5 * rng.standard_normal(H)))
    if fmt == "fp8":
        q, s = oracle.quantize_tokens_fp8(x)
        return q, s, ops.fp8_values(q, s)
    q, s = ops.quantize_mxfp4(x)
    return q, s, ops.mxfp4_values(q, s)


def check(got, y, mag, H, gated):
    """got bf16 bits [R, O]; y, mag of the oracle (NaN where untouched)."""
    mine = ~np.isnan(y)
    assert np.all(got[~mine] == SENT_BF16), "rows of no expert were written"
    v = (got.astype(np.uint32) << 16).view(np.float32).astype(np.float64)
    err = H * 2.0 ** -23 * mag + (2.0 ** -19 * np.abs(y) if gated else 0)
    bad = mine & ~(np.abs(v - y) <= err + 2.0 ** -8 * (np.abs(y) + err) + 2.0 ** -133)
    assert not bad.any(), "%d of %d off, first %s: got %r want %r" % (
        bad.sum(), mine.sum(), np.argwhere(bad)[0].tolist(), v[bad][0], y[bad][0])


def run(ep, counts, H, N, fmt, gated, capacity=0, extra=0, seed=0, stream=None):
    """extra: rows behind the last expert (packed)."""
    print("case product", counts if len(counts) < 12 else (len(counts), max(counts)), H, N, fmt, gated, capacity, extra, flush=True)
    rng = np.random.default_rng(seed)
    E = len(counts)
    rows = E * capacity if capacity else sum(counts) + extra
    q, s, a = rows_of(rng, rows, H, fmt)
    wq, ws, w = rows_of(rng, E * N, H, "mxfp4")
    first = [e * capacity for e in range(E)] if capacity else np.concatenate([[0], np.cumsum(counts)]).tolist()
    y, mag = ops.expert_product(a, w.reshape(E, N, H), list(zip(first, counts)), gated)
    er = np.array(counts if capacity else first, dtype=np.int32)
    out = torch.full((rows, N // 2 if gated else N), SENT_BF16, dtype=torch.int16, device="cuda")
    ep.ep_expert_product(to_dev(q), to_dev(s), ep.EP_RECV_FP8_E4M3_G128 if fmt == "fp8" else ep.EP_RECV_MXFP4_G32,
                         to_dev(wq).view(E, N, H // 2), to_dev(ws).view(E, N, H // 32), to_dev(er), capacity,
                         ep.EP_ACT_SWIGLU if gated else ep.EP_ACT_NONE, out)
    torch.cuda.synchronize()
    check(out.cpu().numpy().view(np.uint16), y, mag, H, gated)


COUNTS = [[1], [0, 3, 0], [16, 17, 15, 0, 1, 33], [64, 65, 63], [128, 0, 129, 127, 5], [257, 1, 300], [0, 0, 0, 40]]


@pytest.mark.parametrize("fmt", ["mxfp4", "fp8"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("H,N", [(128, 16), (384, 64), (640, 208), (1152, 528), (512, 256)])
def test_product(gpu, counts, H, N, fmt, gated):
    run(gpu, counts, H, N, fmt, gated, extra=3, seed=H + N)


@pytest.mark.parametrize("fmt", ["mxfp4", "fp8"])
@pytest.mark.parametrize("H,N", [(256, 8), (896, 24), (128, 1000), (2048, 136)])
def test_product_narrow(gpu, H, N, fmt):
    """Channel counts that are multiples of 8 only."""
    run(gpu, [3, 0, 70, 1], H, N, fmt, False, extra=1)


@pytest.mark.parametrize("fmt", ["mxfp4", "fp8"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("counts,capacity", [([0, 5, 1, 9], 9), ([128, 3, 0], 128), ([40, 33], 47), ([1, 1, 1, 0, 1], 1)])
def test_product_padded(gpu, counts, capacity, fmt, gated):
    run(gpu, counts, 768, 160, fmt, gated, capacity=capacity)


@pytest.mark.parametrize("fmt", ["mxfp4", "fp8"])
def test_product_many_experts(gpu, fmt):
    rng = np.random.default_rng(1)
    run(gpu, rng.integers(0, 3, 1024).tolist(), 128, 32, fmt, False)
    run(gpu, (rng.integers(0, 40, 100) * (rng.random(100) < 0.5)).astype(int).tolist(), 256, 96, fmt, True)


@pytest.mark.parametrize("fmt", ["mxfp4", "fp8"])
@pytest.mark.parametrize("gated", [False, True])
def test_product_large_rows(gpu, fmt, gated):
    """Enough rows per expert for the largest tiles, with ragged ends."""
    run(gpu, [515, 260, 1023], 1024, 592, fmt, gated)
    run(gpu, [1, 2000], 7168, 32, fmt, gated)


@pytest.mark.parametrize("fmt", ["mxfp4", "fp8"])
@pytest.mark.parametrize("H", [512, 640, 1280])
@pytest.mark.parametrize("experts,rows,N", [(45, 5, 1536), (24, 50, 2816), (12, 130, 5888), (7, 300, 5120)])
def test_product_stages(gpu, experts, rows, N, H, fmt):
    """Rows of two, three and five stages, each tile, several tiles in turn on a workgroup."""
    rng = np.random.default_rng(H)
    counts = rng.integers(0, 2 * rows + 1, experts).tolist()
    run(gpu, counts, H, N, fmt, H % 256 == 0 and N % 512 == 0, seed=H)


def test_product_clamps_bad_spans(gpu):
    """Offsets and counts outside the buffer are clamped to it."""
    ep = gpu
    rng = np.random.default_rng(0)
    q, s, a = rows_of(rng, 40, 256, "mxfp4")
    wq, ws, w = rows_of(rng, 4 * 48, 256, "mxfp4")
    for er, cap, spans in [([-5, 10, 5, 1000, 7], 0, [(0, 10), (10, 0), (5, 35), (40, 0)]),
                           ([99, -3, 10, 2 ** 31 - 1], 10, [(0, 10), (10, 0), (20, 10), (30, 10)]),
                           ([0, 0, 0, 0, 0], 0, [(0, 0)] * 4)]:
        # experts 0 and 2 share rows 5..9 in the first: one of the two writes last
        out = torch.full((40, 48), SENT_BF16, dtype=torch.int16, device="cuda")
        ep.ep_expert_product(to_dev(q), to_dev(s), ep.EP_RECV_MXFP4_G32, to_dev(wq).view(4, 48, 128), to_dev(ws).view(4, 48, 8),
                             to_dev(np.array(er, dtype=np.int32)), cap, ep.EP_ACT_NONE, out)
        torch.cuda.synchronize()
        y, mag = ops.expert_product(a, w.reshape(4, 48, 256), spans, False)
        got = out.cpu().numpy().view(np.uint16)
        if cap == 0 and er[0] == -5:
            got, y, mag = np.delete(got, range(5, 10), 0), np.delete(y, range(5, 10), 0), np.delete(mag, range(5, 10), 0)
        check(got, y, mag, 256, False)


def test_product_scales_and_nan(gpu):
    """Scales from 2^-127 on; a NaN scale makes its row's sums NaN and no
    other's."""
    ep = gpu
    rng = np.random.default_rng(5)
    H, N = 256, 32
    q, s, _ = rows_of(rng, 8, H, "mxfp4")
    wq, ws, _ = rows_of(rng, N, H, "mxfp4")
    s[1] = 0
    s[2, 3] = 255
    s[3] = 180
    ws[4] = 60
    ws[5, 1] = 255
    y, mag = ops.expert_product(ops.mxfp4_values(q, s), ops.mxfp4_values(wq, ws)[None], [(0, 8)], False)
    out = torch.empty(8, N, dtype=torch.bfloat16, device="cuda")
    ep.ep_expert_product(to_dev(q), to_dev(s), ep.EP_RECV_MXFP4_G32, to_dev(wq)[None], to_dev(ws)[None],
                         to_dev(np.array([0, 8], dtype=np.int32)), 0, ep.EP_ACT_NONE, out)
    v = out.double().cpu().numpy()
    nan = np.zeros((8, N), dtype=bool)
    nan[2], nan[:, 5] = True, True
    assert np.array_equal(np.isnan(v), nan)
    err = H * 2.0 ** -23 * mag
    assert np.all((np.abs(v - y) <= err + 2.0 ** -8 * (np.abs(y) + err) + 2.0 ** -126)[~nan])


def test_product_repeats_bitwise_on_streams_and_in_graphs(gpu):
    """The same bits on every run: on two side streams at once, and captured
    and replayed between eager calls."""
    ep = gpu
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    E, H, N = 8, 1024, 512
    counts = [3, 0, 200, 17, 64, 1, 130, 40]
    off = torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32, device="cuda")
    R = sum(counts)
    a, s = ep.quantize_rows(torch.randn(R, H, generator=g, device="cuda").bfloat16())
    w, ws = ep.quantize_rows(torch.randn(E * N, H, generator=g, device="cuda").bfloat16())
    w, ws = w.view(E, N, -1), ws.view(E, N, -1)
    h = ep.Handle(None, off, None, None, E)
    want = ep.expert_product(a, s, w, ws, h, ep.EP_ACT_SWIGLU)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = []
    for _ in range(4):
        for st in streams:
            with torch.cuda.stream(st):
                outs.append(ep.expert_product(a, s, w, ws, h, ep.EP_ACT_SWIGLU))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=streams[0]):
        y = ep.expert_product(a, s, w, ws, h, ep.EP_ACT_SWIGLU)
    for k in range(3):
        a.copy_(a.roll(1, 0))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        eager = ep.expert_product(a, s, w, ws, h, ep.EP_ACT_SWIGLU)
        torch.cuda.synchronize()
        assert torch.equal(y, eager)


def test_product_empty(gpu):
    ep = gpu
    h = ep.Handle(None, torch.zeros(3, dtype=torch.int32, device="cuda"), None, None, 2)
    z = lambda *n: torch.zeros(n, dtype=torch.uint8, device="cuda")
    assert ep.expert_product(z(0, 64), z(0, 4), z(2, 16, 64), z(2, 16, 4), h).shape == (0, 16)


def test_product_refuses_mismatched_shapes(gpu):
    ep = gpu
    z = lambda *n: torch.zeros(n, dtype=torch.uint8, device="cuda")
    h = ep.Handle(None, torch.zeros(3, dtype=torch.int32, device="cuda"), None, None, 2)
    with pytest.raises(ValueError):
        ep.expert_product(z(4, 32), z(4, 4), z(2, 16, 64), z(2, 16, 4), h)
    with pytest.raises(ValueError):
        ep.expert_product(z(4, 64), z(4, 4), z(2, 20, 64), z(2, 20, 4), h)
    with pytest.raises(ValueError):
        ep.expert_product(z(4, 64), z(4, 4), z(3, 16, 64), z(3, 16, 4), h)
    with pytest.raises(ValueError):
        ep.expert_product(z(4, 96), z(4, 6), z(2, 16, 96), z(2, 16, 6), h)


@pytest.mark.parametrize("fmt", ["mxfp4", "fp8"])
@pytest.mark.parametrize("H", [512, 896])
def test_product_clamps_bad_spans_in_tiles(gpu, H, fmt):
    """Offsets and counts outside the buffer, at sizes that go in tiles."""
    ep = gpu
    rng = np.random.default_rng(H)
    q, s, a = rows_of(rng, 400, H, fmt)
    wq, ws, w = rows_of(rng, 4 * 48, H, "mxfp4")
    for er, cap, spans in [([-5, 100, 50, 100000, 7], 0, [(0, 100), (100, 0), (50, 350), (400, 0)]),
                           ([2 ** 31 - 1, -2 ** 31, 3, 3, 3], 0, [(400, 0), (0, 3), (3, 0), (3, 0)]),
                           ([999, -3, 100, 2 ** 31 - 1], 100, [(0, 100), (100, 0), (200, 100), (300, 100)])]:
        out = torch.full((400, 48), SENT_BF16, dtype=torch.int16, device="cuda")
        print("case spans", H, fmt, er, cap, flush=True)
        ep.ep_expert_product(to_dev(q), to_dev(s), ep.EP_RECV_FP8_E4M3_G128 if fmt == "fp8" else ep.EP_RECV_MXFP4_G32,
                             to_dev(wq).view(4, 48, H // 2), to_dev(ws).view(4, 48, H // 32),
                             to_dev(np.array(er, dtype=np.int32)), cap, ep.EP_ACT_NONE, out)
        torch.cuda.synchronize()
        y, mag = ops.expert_product(a, w.reshape(4, 48, H), spans, False)
        got = out.cpu().numpy().view(np.uint16)
        if er[0] == -5:  # experts 0 and 2 share rows 50..99: one of the two writes last
            got, y, mag = [np.delete(v, range(50, 100), 0) for v in (got, y, mag)]
        check(got, y, mag, H, False)


@pytest.mark.parametrize("fmt", ["mxfp4", "fp8"])
@pytest.mark.parametrize("H", [640, 1024])
def test_product_nan_stays_in_its_row_and_channel_in_tiles(gpu, H, fmt):
    """A NaN scale (or FP8 code) makes its row's sums NaN, one of the weights'
    its channel's, and no others."""
    ep = gpu
    rng = np.random.default_rng(H)
    N = 96
    q, s, _ = rows_of(rng, 70, H, fmt)
    wq, ws, _ = rows_of(rng, N, H, "mxfp4")
    if fmt == "fp8":
        q[2, H - 3], q[40, 5] = 0x7F, 0xFF
        a = ops.fp8_values(q, s)
    else:
        s[2, H // 32 - 1], s[40, 0] = 255, 255
        a = ops.mxfp4_values(q, s)
    ws[5, 1], ws[77, H // 32 - 1] = 255, 255
    y, mag = ops.expert_product(a, ops.mxfp4_values(wq, ws)[None], [(0, 70)], False)
    out = torch.empty(70, N, dtype=torch.bfloat16, device="cuda")
    ep.ep_expert_product(to_dev(q), to_dev(s), ep.EP_RECV_FP8_E4M3_G128 if fmt == "fp8" else ep.EP_RECV_MXFP4_G32,
                         to_dev(wq)[None], to_dev(ws)[None], to_dev(np.array([0, 70], dtype=np.int32)), 0,
                         ep.EP_ACT_NONE, out)
    v = out.double().cpu().numpy()
    nan = np.zeros((70, N), dtype=bool)
    nan[[2, 40]], nan[:, [5, 77]] = True, True
    assert np.array_equal(np.isnan(v), nan)
    err = H * 2.0 ** -23 * mag
    assert np.all((np.abs(v - y) <= err + 2.0 ** -8 * (np.abs(y) + err) + 2.0 ** -126)[~nan])


@pytest.mark.parametrize("fmt", ["mxfp4", "fp8"])
def test_product_offsets_beyond_32_bits(gpu, fmt):
    """Rows and weights that lie more than 2^32 bytes into their buffers."""
    ep = gpu
    rng = np.random.default_rng(3)
    H, N, E, R, n = 32768, 272, 1000, 270000, 37
    q, s, a = rows_of(rng, n, H, fmt)
    wq, ws, w = rows_of(rng, N, H, "mxfp4")
    row, scale = (H, H // 128) if fmt == "fp8" else (H // 2, H // 32)
    dq = torch.zeros(R, row, dtype=torch.uint8, device="cuda")
    ds = torch.zeros(R, scale, dtype=torch.float32 if fmt == "fp8" else torch.uint8, device="cuda")
    dw = torch.zeros(E, N, H // 2, dtype=torch.uint8, device="cuda")
    dws = torch.zeros(E, N, H // 32, dtype=torch.uint8, device="cuda")
    assert dq.numel() > 2 ** 32 and dw.numel() > 2 ** 32
    dq[R - n:], ds[R - n:], dw[E - 1], dws[E - 1] = to_dev(q), to_dev(s), to_dev(wq), to_dev(ws)
    off = torch.full((E + 1,), R - n, dtype=torch.int32, device="cuda")
    off[E] = R
    out = torch.full((R, N), SENT_BF16, dtype=torch.int16, device="cuda")
    ep.ep_expert_product(dq, ds, ep.EP_RECV_FP8_E4M3_G128 if fmt == "fp8" else ep.EP_RECV_MXFP4_G32, dw, dws, off, 0,
                         ep.EP_ACT_NONE, out)
    torch.cuda.synchronize()
    y, mag = ops.expert_product(a, w[None], [(0, n)], False)
    check(out[R - n:].cpu().numpy().view(np.uint16), y, mag, H, False)
    assert bool((out[:R - n] == SENT_BF16).all())
