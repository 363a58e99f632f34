"""Every tile of the experts' bf16 layers: sizes that the choice of tile sends
to each of them (on 256 CUs), with several tiles in turn on a workgroup and
ragged ends, on whole numbers, whose sums are exact."""

import numpy as np
import pytest
import torch

from tests.test_expert_linear_gpu import Rows, backward, forward, weights

pytestmark = pytest.mark.gpu


def ragged(experts, rows, seed):
    rng = np.random.default_rng(seed)
    counts = rng.integers(rows // 2, rows + rows // 2 + 1, experts)
    counts[1] = 0
    return counts.tolist()


# rows (dense, or experts and mean rows), channels of the result
TILES = {"256x256 dense": (4100, 4400), "256x256": ((8, 560), 4400), "192x256": ((70, 135), 1304), "128x256": ((70, 55), 1304),
         "128x256 dense": (1100, 8000), "128x128": (600, 6400), "64x128": ((70, 7), 704), "64x128 dense": (500, 3800),
         "64x128 of 352": (700, 4000), "64x128 in groups, more than CUs": ((20, 75), 1240),
         "64x64": (40, 1000), "64x64, more than CUs": ((20, 75), 600), "few rows": (13, 1000), "few rows of few experts": ((5, 3), 200)}


def rows_of(rows):
    return Rows(rows if isinstance(rows, int) else ragged(*rows, seed=rows[1]), extra=0 if isinstance(rows, int) else 5)


@pytest.mark.parametrize("C", [56, 448, 1000])
@pytest.mark.parametrize("tile", TILES)
def test_linear_tiles(gpu, tile, C):
    rows, O = TILES[tile]
    r = rows_of(rows)
    forward(gpu, r, C, O, bias=True, residual=True)
    forward(gpu, r, C, 16 * (O // 16), gated=True, save=C == 448, bias=C == 56, whole=C != 1000)


@pytest.mark.parametrize("rows,O", [(500, 3800), ((20, 75), 1240)], ids=["dense", "more than CUs"])
def test_linear_long_sums_in_groups(gpu, rows, O):
    r = rows_of(rows)
    forward(gpu, r, 2056, O, bias=True, residual=True)
    forward(gpu, r, 2056, O // 16 * 16, gated=True, save=True, whole=False)


@pytest.mark.parametrize("C", [56, 448, 1000])
@pytest.mark.parametrize("tile", TILES)
def test_backward_tiles(gpu, tile, C):
    rows, O = TILES[tile]
    r = rows_of(rows)
    backward(gpu, r, O, C)
    backward(gpu, r, O, C, gated=True, whole=C != 1000)


@pytest.mark.parametrize("counts,H,N", [([700, 0, 1, 450, 900], 1800, 2304), ([401, 830], 3000, 2904),  # 256 x 256
                                        (70, 600, 704), ([3] * 40 + [0, 200], 400, 904),                 # 128 x 256
                                        (5000, 304, 200), ([64, 0, 70], 136, 520)],                      # 128 x 128
                         ids=lambda c: str(c) if isinstance(c, int) else "x".join(map(str, c[:3])))
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_weights_tiles(gpu, counts, H, N, dtype):
    r = Rows(ragged(70, counts, 1) if counts == 70 else counts)
    weights(gpu, r, H, N, dtype=dtype)
    weights(gpu, r, H, N, dtype=dtype, accumulate=True, bias=dtype == torch.float32)


@pytest.mark.parametrize("capacity", [20, 200])
def test_padded_tiles(gpu, capacity):
    rng = np.random.default_rng(capacity)
    r = Rows(rng.integers(0, capacity + 1, 80).tolist(), capacity)
    forward(gpu, r, 264, 1040, gated=True, bias=True, residual=True, save=True)
    backward(gpu, r, 1040, 264)
    weights(gpu, r, 264, 136)


def test_sorted_experts(gpu):
    """1024 experts of the most different numbers of rows, ties among them."""
    rng = np.random.default_rng(9)
    counts = (rng.integers(0, 6, 1024) ** 3 * (rng.random(1024) < 0.4)).astype(int).tolist()
    weights(gpu, Rows(counts), 136, 144, dtype=torch.float32)
    weights(gpu, Rows(counts, capacity=125), 136, 144)


def test_tiles_in_graphs_and_at_once(gpu):
    """The largest tiles, captured and replayed between eager calls, and twice at once."""
    ep = gpu
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    new = lambda *shape: torch.randn(*shape, generator=g, device="cuda").bfloat16()
    E, H, N = 8, 512, 4400
    off = torch.tensor(np.concatenate([[0], np.cumsum(ragged(E, 560, 3))]).astype(np.int32)).cuda()
    R = int(off[-1])
    a, w, go, mid = new(R, H), new(E, N, H), new(R, H), new(R, 2 * N)
    w2 = new(E, H, N)
    h = ep.Handle(None, off, None, None, E)

    def step():
        return (ep.expert_linear(a, w, h), ep.expert_linear_backward(go, w2, h, p=mid), *ep.expert_linear_backward_weights(go, a, h, bias=True))

    want = step()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = []
    for st in streams * 2:
        with torch.cuda.stream(st):
            outs.append(step())
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for o in outs for x, y in zip(o, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=streams[0]):
        y = step()
    for _ in range(3):
        a.copy_(a.roll(1, 0))
        go.copy_(go.roll(3, 0))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        eager = step()
        torch.cuda.synchronize()
        assert all(torch.equal(x, z) for x, z in zip(y, eager))
