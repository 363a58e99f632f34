"""ep_expert_product on sums that binary32 holds exactly, in any order.

Codes are small multiples of a power of two and every scale is a power of
two, so that the sum of the magnitudes of a row's products is below 2^24
times their common unit (asserted): each partial sum is exact in binary32,
whatever the order, and y must be BF16_RNE of the exact sum, bit for bit.  A
lost, doubled or misplaced channel shows, at any length.  With the gated
activation u and g are exact and y is within |g| 2^-22 + 2^-20 of silu(g) u
relatively (the exponential's argument off by half a unit of its last place,
twice that of its result, one division, two more roundings), and half a step
of BF16, 2^-8 of the value.

FP8 rows carry codes of 256 among codes below 1: their products lie up to 15
binades apart, more than the matrix unit keeps of eight neighbouring
channels."""

import numpy as np
import pytest
import torch

from tests.gpu_run import SENT_BF16

pytestmark = pytest.mark.gpu

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def codes4(g, rows, H, low, high):
    """Random E2M1 codes, scale bytes in [low, high] -> (q, scale, values in binary64, their unit)."""
    q = torch.randint(0, 256, (rows, H // 2), generator=g, device="cuda", dtype=torch.uint8)
    s = torch.randint(low, high + 1, (rows, H // 32), generator=g, device="cuda", dtype=torch.uint8)
    grid = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float64, device="cuda")
    v = torch.stack([grid[(q & 15).int()], grid[(q >> 4).int()]], -1).view(rows, H // 32, 32)
    return q, s, (v * torch.exp2(s.double() - 127).unsqueeze(-1)).view(rows, H), 0.5 * 2.0 ** (low - 127)


def codes8(g, rows, H, every):
    """E4M3 codes: 256 in one channel of ``every``, else multiples of 2^-4 below 1; scales 1 and 2."""
    v = torch.randint(-15, 16, (rows, H), generator=g, device="cuda").double() / 16
    at = torch.randint(0, every, (rows, H // every, 1), generator=g, device="cuda")
    sign = torch.randint(0, 2, (rows, H // every, 1), generator=g, device="cuda").double() * 2 - 1
    v = v.view(rows, H // every, every).scatter(2, at, 256 * sign).view(rows, H)
    q = v.float().to(torch.float8_e4m3fn)
    assert torch.equal(q.double(), v)
    s = torch.randint(0, 2, (rows, H // 128), generator=g, device="cuda").float() + 1
    return q.view(torch.uint8), s, (v.view(rows, H // 128, 128) * s.double().unsqueeze(-1)).view(rows, H), 2.0 ** -4


def run(ep, counts, H, N, fmt, gated, capacity=0, extra=3, every=8, seed=0):
    print("case exact", len(counts), sum(counts), H, N, fmt, gated, capacity, flush=True)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + H)
    E, O = len(counts), N // 2 if gated else N
    rows = E * capacity if capacity else sum(counts) + extra
    a, s, av, unit_a = codes8(g, rows, H, every) if fmt == "fp8" else codes4(g, rows, H, 127, 129)
    wq, ws, wv, unit_w = codes4(g, E * N, H, 114, 115)
    first = [e * capacity for e in range(E)] if capacity else np.concatenate([[0], np.cumsum(counts)]).tolist()
    er = torch.tensor(counts if capacity else first, dtype=torch.int32, device="cuda")
    y = torch.full((rows, O), SENT_BF16, dtype=torch.int16, device="cuda")
    ep.ep_expert_product(a, s, ep.EP_RECV_FP8_E4M3_G128 if fmt == "fp8" else ep.EP_RECV_MXFP4_G32, wq.view(E, N, -1),
                         ws.view(E, N, -1), er, capacity, ep.EP_ACT_SWIGLU if gated else ep.EP_ACT_NONE, y)
    torch.cuda.synchronize()
    mine = torch.zeros(rows, dtype=torch.bool, device="cuda")
    wv = wv.view(E, N, H)
    for e, n in enumerate(counts):
        if n == 0:
            continue
        r = slice(first[e], first[e] + n)
        mine[r] = True
        wt = wv[e].t().contiguous()
        p = av[r] @ wt
        if n <= 64:  # (the same distributions in every row)
            assert float((av[r].abs() @ wt.abs()).max()) < 2.0 ** 24 * unit_a * unit_w
        got = y[r].view(torch.bfloat16)
        if not gated:
            assert torch.equal(p.float().double(), p)
            assert torch.equal(got, p.float().bfloat16()), (e, n, int((got != p.float().bfloat16()).sum()))
            continue
        gate, up = p[:, :O], p[:, O:]
        want = gate * torch.sigmoid(gate) * up
        err = want.abs() * (gate.abs() * 2.0 ** -22 + 2.0 ** -20)
        bad = ~((got.double() - want).abs() <= err + 2.0 ** -8 * (want.abs() + err) + 2.0 ** -133)
        assert not bad.any(), (e, n, int(bad.sum()), got[bad][:4], want[bad][:4])
    assert bool((y[~mine] == SENT_BF16).all()), "rows of no expert were written"


@pytest.mark.parametrize("fmt", ["mxfp4", "fp8"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("H", [128, 256, 384, 512, 640, 1152])
def test_exact_sums(gpu, H, gated, fmt):
    run(gpu, [5, 0, 33, 64, 1], H, 272, fmt, gated)


@pytest.mark.parametrize("fmt", ["mxfp4", "fp8"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("counts", [[3, 0, 70], [400, 17]], ids=["few", "many"])
@pytest.mark.parametrize("H,every", [(7168, 64), (32768, 512)])
def test_exact_long_sums(gpu, H, every, counts, gated, fmt):
    run(gpu, counts, H, 80, fmt, gated, every=every)


@pytest.mark.parametrize("fmt", ["mxfp4", "fp8"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("H", [512, 640, 1024, 1280, 1536, 1792, 3328, 7168])
@pytest.mark.parametrize("experts,rows,N", [(45, 5, 2048), (24, 50, 3328), (12, 130, 5888), (7, 400, 7168)])
def test_exact_sums_over_several_tiles(gpu, experts, rows, N, H, gated, fmt):
    """Every kernel of each format, with and without the activation, on more
    tiles than workgroups: copies that run on into the next tile, after 2, 3,
    4, 5, 6, 7, 13 and 28 stages, the last one half in some."""
    counts = np.random.default_rng(experts + H).integers(0, 2 * rows + 1, experts).tolist()
    run(gpu, counts, H, N, fmt, gated, every=8 if H < 1200 else 64, seed=rows)


@pytest.mark.parametrize("fmt", ["mxfp4", "fp8"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("counts,capacity", [([7, 0, 96, 33], 96), ([300, 1, 257, 0, 64], 300)])
@pytest.mark.parametrize("H", [256, 1024])
def test_exact_sums_padded(gpu, counts, capacity, H, gated, fmt):
    run(gpu, counts, H, 1040, fmt, gated, capacity=capacity)


@pytest.mark.parametrize("counts", [[40], [9, 0, 15, 20], [400]], ids=["kernel", "few", "many"])
@pytest.mark.parametrize("H", [128, 384, 512, 896, 2048])
def test_every_fp8_code(gpu, counts, H):
    """All finite codes side by side.  Not exact: 128
    channels are at most 4 matrix instructions of 8 additions, then a scaled
    addition to the sum so far, so (33 + H / 128) 2^-24 of the magnitudes, and
    half a step of BF16."""
    ep, N, E = gpu, 96, len(counts)
    g = torch.Generator(device="cuda")
    g.manual_seed(H)
    rows = sum(counts)
    q = torch.randint(0, 256, (rows, H), generator=g, device="cuda", dtype=torch.uint8)
    q = torch.where((q & 0x7F) == 0x7F, q ^ 1, q)
    s = torch.rand(rows, H // 128, generator=g, device="cuda") + 0.5
    wq, ws, wv, _ = codes4(g, E * N, H, 124, 130)
    av = (q.view(torch.float8_e4m3fn).double().view(rows, -1, 128) * s.double().unsqueeze(-1)).view(rows, H)
    first = np.concatenate([[0], np.cumsum(counts)]).tolist()
    y = torch.empty(rows, N, dtype=torch.bfloat16, device="cuda")
    print("case every code", counts, H, flush=True)
    ep.ep_expert_product(q, s, ep.EP_RECV_FP8_E4M3_G128, wq.view(E, N, -1), ws.view(E, N, -1),
                         torch.tensor(first, dtype=torch.int32, device="cuda"), 0, ep.EP_ACT_NONE, y)
    for e, n in enumerate(counts):
        r, wt = slice(first[e], first[e] + n), wv.view(E, N, H)[e].t().contiguous()
        p, m = av[r] @ wt, av[r].abs() @ wt.abs()
        err = (33 + H / 128) * 2.0 ** -24 * m
        assert bool(((y[r].double() - p).abs() <= err + 2.0 ** -8 * (p.abs() + err)).all())


@pytest.mark.parametrize("fmt", ["mxfp4", "fp8"])
def test_largest_matrix(gpu, fmt):
    """65536 channels in and out: 2^31 bytes of one expert's weights, of which
    a few rows are not zero."""
    ep, H, N, n, at = gpu, 65536, 65536, 5, [0, 1, 4095, 32767, 32768, 65400, 65535]
    g = torch.Generator(device="cuda")
    g.manual_seed(9)
    a, s, av, unit_a = codes8(g, n, H, 1024) if fmt == "fp8" else codes4(g, n, H, 127, 128)
    wq, ws, wv, unit_w = codes4(g, len(at), H, 120, 120)
    w = torch.zeros(1, N, H // 2, dtype=torch.uint8, device="cuda")
    scale = torch.full((1, N, H // 32), 127, dtype=torch.uint8, device="cuda")
    w[0, at], scale[0, at] = wq, ws
    y = torch.empty(n, N, dtype=torch.bfloat16, device="cuda")
    print("case largest matrix", fmt, flush=True)
    ep.ep_expert_product(a, s, ep.EP_RECV_FP8_E4M3_G128 if fmt == "fp8" else ep.EP_RECV_MXFP4_G32, w, scale,
                         torch.tensor([0, n], dtype=torch.int32, device="cuda"), 0, ep.EP_ACT_NONE, y)
    torch.cuda.synchronize()
    assert float((av.abs() @ wv.abs().t().contiguous()).max()) < 2.0 ** 24 * unit_a * unit_w
    want = torch.zeros(n, N, dtype=torch.bfloat16, device="cuda")
    want[:, at] = (av @ wv.t().contiguous()).float().bfloat16()
    assert torch.equal(y, want)
