"""Quantised rows: ep_quantize_rows, ep_dequantize_rows and the MXFP4
dispatch, bit for bit against the oracle."""

import numpy as np
import pytest
import torch

import oracle
from oracle import operators as ops
from tests.gpu_run import SENT_F32, SENT_I32, SENT_U8, host, to_dev
from workloads import make_workload

pytestmark = pytest.mark.gpu


def bits_of(rows, H, seed):
    """Rows of channels of unequal size, with zero groups, tiny and huge
    groups, signed zeros and ties."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((rows, H)).astype(np.float32) * np.exp(2 * rng.standard_normal(H)).astype(np.float32)
    x = x.reshape(rows, -1, 32)
    kind = rng.random(x.shape[:2])
    x[kind < 0.05] = 0.0
    x[(kind >= 0.05) & (kind < 0.1)] *= 2.0 ** -126
    x[(kind >= 0.1) & (kind < 0.15)] *= 2.0 ** 100
    ties = (kind >= 0.15) & (kind < 0.3)
    x[ties] = rng.integers(-28, 29, x[ties].shape) * 0.25
    x[(kind >= 0.3) & (kind < 0.35)] *= -0.0
    t = torch.from_numpy(x.reshape(rows, H)).to(torch.bfloat16)
    return t.view(torch.int16).numpy().view(np.uint16)


@pytest.mark.parametrize("rows,H", [(1, 32), (3, 64), (17, 96), (130, 256), (5, 7168), (1000, 288), (2049, 2048)])
def test_quantize_mxfp4(gpu, rows, H):
    ep = gpu
    print("case quantize mxfp4", rows, H, flush=True)
    x = bits_of(rows, H, rows + H)
    q = torch.full((rows + 1, H // 2), SENT_U8, dtype=torch.uint8, device="cuda")
    s = torch.full((rows + 1, H // 32), SENT_U8, dtype=torch.uint8, device="cuda")
    ep.ep_quantize_rows(to_dev(x.view(np.int16)), ep.EP_RECV_MXFP4_G32, q[:rows], s[:rows])
    wq, ws = ops.quantize_mxfp4(x)
    assert np.array_equal(host(q)[:rows], wq) and np.array_equal(host(s)[:rows], ws)
    assert np.all(host(q)[rows] == SENT_U8) and np.all(host(s)[rows] == SENT_U8)
    v = ep.dequantize_rows(q[:rows], s[:rows])
    want = ops.mxfp4_values(wq, ws)
    assert np.array_equal(v.double().cpu().numpy(), want)
    assert np.array_equal(np.signbit(v.double().cpu().numpy()), np.signbit(want))


def test_quantize_every_bf16_value(gpu):
    """Every finite BF16 value beside a group maximum at which it is a code of
    its own, infinities and NaN in groups of their own."""
    ep = gpu
    v = np.arange(65536, dtype=np.uint32).astype(np.uint16)
    x = np.zeros((65536, 32), dtype=np.uint16)
    x[:, 0] = v  # alone in its group
    x[:, 40 % 32] = 0
    y = np.zeros((65536, 32), dtype=np.uint16)
    mag = v & 0x7FFF
    y[:, 3] = v
    y[:, 7] = np.minimum(mag + 0x80, 0x7F7F)  # the maximum, one binade above
    z = np.zeros((65536, 32), dtype=np.uint16)
    z[:, 31] = v
    z[:, 0] = np.minimum(mag + 0x180, 0x7F7F)
    for rows in (x, y, z):
        q, s = ep.quantize_rows(to_dev(rows.view(np.int16)))
        wq, ws = ops.quantize_mxfp4(rows)
        assert np.array_equal(host(s), ws)
        assert np.array_equal(host(q), wq)


def test_dequantize_every_code_and_scale(gpu):
    ep = gpu
    q = np.tile(np.arange(256, dtype=np.uint8), (256, 1))  # 512 channels, every byte
    s = np.repeat(np.arange(256, dtype=np.uint8)[:, None], 16, axis=1)
    v = ep.dequantize_rows(to_dev(q), to_dev(s)).double().cpu().numpy()
    want = ops.mxfp4_values(q, s)
    want = np.where(np.abs(want) >= 2.0 ** 128, np.sign(want) * np.inf, want)  # beyond BF16's range
    assert np.array_equal(v, want, equal_nan=True)


@pytest.mark.parametrize("rows,H", [(1, 128), (37, 256), (5, 7168), (1001, 384)])
def test_quantize_fp8(gpu, rows, H):
    """The dispatch's FP8 codes and scales, on rows in their own order."""
    ep = gpu
    rng = np.random.default_rng(rows)
    x = torch.from_numpy(rng.standard_normal((rows, H)).astype(np.float32)).to(torch.bfloat16)
    x = x.view(torch.int16).numpy().view(np.uint16)
    x[:, :128] = 0
    q, s = ep.quantize_rows(to_dev(x.view(np.int16)), ep.EP_RECV_FP8_E4M3_G128)
    wq, ws = oracle.quantize_tokens_fp8(x)
    assert np.array_equal(host(q), wq) and np.array_equal(host(s), ws)
    v = ep.dequantize_rows(q, s, ep.EP_RECV_FP8_E4M3_G128)
    want = torch.from_numpy(ops.fp8_values(wq, ws).astype(np.float32)).to(torch.bfloat16)  # one binary32 product, rounded to BF16
    assert torch.equal(v.cpu(), want)


def test_dequantize_every_fp8_code(gpu):
    ep = gpu
    q = np.tile(np.arange(256, dtype=np.uint8), (4, 2))
    s = np.array([[1.0, 0.3, 2.0 ** -126, 1e30]] * 4, dtype=np.float32)
    v = ep.dequantize_rows(to_dev(q), to_dev(s), ep.EP_RECV_FP8_E4M3_G128)
    with np.errstate(over="ignore"):
        f = (oracle.e4m3_to_f32(q) * np.repeat(s, 128, axis=1)).astype(np.float32)
    want = torch.from_numpy(f).to(torch.bfloat16)
    assert torch.equal(torch.isnan(v).cpu(), torch.isnan(want))
    assert torch.equal(torch.nan_to_num(v.cpu()), torch.nan_to_num(want))


def check_dispatch(ep, wl, capacity, how):
    T, H, K, E = wl.T, wl.H, wl.K, wl.E
    print("case mxfp4 dispatch", T, H, K, E, capacity, how, flush=True)
    rows = E * capacity if capacity else T * K
    x, idx, w = to_dev(wl.x_bits.view(np.int16)), to_dev(wl.topk_idx), to_dev(wl.topk_weights)
    if how == "int64":
        idx = idx.long()
    new = lambda n, d=torch.int32, fill=SENT_I32: torch.full((n,), fill, dtype=d, device="cuda")
    counts, offsets, src = new(E), None if capacity else new(E + 1), new(rows)
    slot = torch.full((T, K), SENT_I32, dtype=torch.int32, device="cuda")
    q = torch.full((rows, H // 2), SENT_U8, dtype=torch.uint8, device="cuda")
    s = torch.full((rows, H // 32), SENT_U8, dtype=torch.uint8, device="cuda")
    rw = new(rows, torch.float32, SENT_F32)
    fmt = ep.EP_RECV_MXFP4_G32
    if how == "split":
        ep.ep_dispatch_layout(idx, E, counts, offsets, slot, src)
        ep.ep_dispatch(x, slot, w, fmt, q, s, rw)
    elif how == "noalloc":
        ep.ep_layout_dispatch_noalloc(idx, x, w, E, capacity, fmt, counts, offsets, slot, src, q, s, rw)
    else:
        nb = ep.ep_layout_workspace_bytes(T, K, E)
        ws = torch.empty(nb, dtype=torch.uint8, device="cuda") if nb else None
        ep.ep_layout_dispatch(idx, x, w, E, capacity, fmt, counts, offsets, slot, src, q, s, rw, ws)
    if capacity:
        want_counts, want_slot, _ = oracle.dispatch_layout_padded(wl.topk_idx, E, capacity)[:3]
    else:
        want_counts, _, want_slot, _ = oracle.dispatch_layout(wl.topk_idx, E)
    assert np.array_equal(host(counts), want_counts) and np.array_equal(host(slot), want_slot)
    wq, ws_ = ops.quantize_mxfp4(wl.x_bits)
    want_q, want_s = np.full((rows, H // 2), SENT_U8, np.uint8), np.full((rows, H // 32), SENT_U8, np.uint8)
    want_w = np.full(rows, SENT_F32, np.float32)
    for k in range(K):
        r = want_slot[:, k]
        m = r >= 0
        want_q[r[m]], want_s[r[m]], want_w[r[m]] = wq[m], ws_[m], wl.topk_weights[m, k]
    assert np.array_equal(host(q), want_q) and np.array_equal(host(s), want_s)
    assert np.array_equal(host(rw), want_w)


@pytest.mark.parametrize("name,T,H,K,E,capacity,how", [
    ("tiny", 64, 256, 2, 16, 0, "split"), ("tiny", 1, 32, 1, 4, 0, "one"), ("tiny", 7, 96, 3, 16, 0, "one"),
    ("decode", 128, 7168, 8, 256, 0, "one"), ("decode", 128, 7168, 8, 256, 128, "one"), ("decode", 33, 288, 5, 64, 9, "int64"),
    ("skew", 700, 1056, 8, 256, 0, "one"), ("skew", 700, 1056, 8, 256, 16, "noalloc"), ("prefill", 4096, 512, 8, 256, 0, "one"),
    ("decode", 130, 2048, 11, 64, 0, "split"), ("prefill", 9000, 64, 8, 256, 0, "noalloc"), ("prefill", 9000, 64, 8, 256, 0, "int64"),
    ("decode", 5, 4096, 32, 64, 0, "one"), ("prefill", 1200, 7168, 6, 256, 0, "split")])
def test_mxfp4_dispatch(gpu, name, T, H, K, E, capacity, how):
    routing = "softmax" if E % 8 or K > E // 2 else None
    over = dict(T=T, H=H, K=K, E=E)
    if routing or E != 256:
        over["routing"] = "softmax"
    wl = make_workload(name, seed=T, **over)
    wl.topk_idx[T // 3] = -1  # a masked token
    wl.topk_idx[0, 0] = -5
    check_dispatch(gpu, wl, capacity, how)


def test_mxfp4_plan_and_wrappers(gpu):
    """StepPlan and the allocating wrappers give the C call's rows."""
    ep = gpu
    wl = make_workload("decode", seed=3, T=40, H=512)
    x, idx, w = to_dev(wl.x_bits.view(np.int16)).view(torch.bfloat16), to_dev(wl.topk_idx), to_dev(wl.topk_weights)
    fmt = ep.EP_RECV_MXFP4_G32
    q, s, rw, h = ep.dispatch(x, idx, w, wl.E, format=fmt)
    q2, s2, _, _ = ep.dispatch(x, None, w, wl.E, handle=h, format=fmt)
    wq, ws = ops.quantize_mxfp4(wl.x_bits)
    src = host(h.src_token)
    assert np.array_equal(host(q), wq[src]) and np.array_equal(host(s), ws[src])
    assert torch.equal(q, q2) and torch.equal(s, s2)
    for cap in (0, 40):
        plan = ep.StepPlan(idx, w, x, wl.E, capacity=cap, format=fmt)
        plan.recv_x.fill_(0)
        plan.recv_scale.fill_(0)
        plan.layout_dispatch()
        if cap == 0:
            assert torch.equal(plan.recv_x, q) and torch.equal(plan.recv_scale, s)
        lq, ls, cnt, lh = ep.low_latency_dispatch(x, idx, 40, wl.E, format=fmt)
        if cap:
            for e in range(wl.E):
                n = int(cnt[e])
                assert torch.equal(lq[e, :n], plan.recv_x.view(wl.E, cap, -1)[e, :n])
                assert torch.equal(ls[e, :n], plan.recv_scale.view(wl.E, cap, -1)[e, :n])
    with pytest.raises(ValueError, match="hidden"):
        ep.StepPlan(idx, w, torch.zeros(40, 48, dtype=torch.bfloat16, device="cuda"), wl.E, format=fmt)


def test_rows_empty(gpu):
    q, s = gpu.quantize_rows(torch.zeros(0, 64, dtype=torch.bfloat16, device="cuda"))
    assert q.shape == (0, 32) and s.shape == (0, 2) and gpu.dequantize_rows(q, s).shape == (0, 64)
