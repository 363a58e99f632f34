"""Offsets that run back and forth over the whole buffer: where the tiles would
reach 2^30 nothing is written."""

import pytest
import torch

from tests.test_expert_linear_gpu import SENT, sentinel

pytestmark = pytest.mark.gpu


def test_too_many_tiles_write_nothing(gpu):
    ep = gpu
    R, E, wide = 1 << 29, 1024, 24  # 512 experts of all the rows: 2^30 tiles of 256
    off = torch.tensor([0, R] * (E // 2) + [0], dtype=torch.int32, device="cuda")
    rows, w = torch.zeros(R, 8, dtype=torch.bfloat16, device="cuda"), torch.zeros(E, wide, 8, dtype=torch.bfloat16, device="cuda")
    out = sentinel(R, wide)
    print("case offsets over all rows", flush=True)
    ep.ep_expert_linear(rows, w, off, 0, ep.EP_ACT_NONE, out)
    torch.cuda.synchronize()
    ep.ep_expert_linear_backward(rows, w.transpose(1, 2).contiguous(), off, 0, out)
    torch.cuda.synchronize()
    for part in out.view(torch.int16).split(1 << 26):
        assert bool((part == SENT).all())
