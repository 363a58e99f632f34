"""Which device a call is launched on, without a GPU: tensors that say they
are on device 0 or 1, and an entry point that records the device that is
current and the stream it is handed."""

import contextlib
import types

import pytest
import torch

T, K, E, H, CAP = 4, 2, 8, 128, 4


class OnGpu(torch.Tensor):
    """A host tensor that reports a GPU's device."""

    index = 0
    is_cuda = True
    device = property(lambda self: "cuda:%d" % self.index)

    def get_device(self):
        return self.index


class OnGpu1(OnGpu):
    index = 1


@pytest.fixture
def ep(monkeypatch):
    import combine_ep_dispatch_amd as ep
    from combine_ep_dispatch_amd import api

    current, calls = [0], []

    @contextlib.contextmanager
    def device(i):
        old, current[0] = current[0], i
        yield
        current[0] = old

    class Lib:
        def __getattr__(self, name):
            return lambda *a: calls.append((name, current[0], a[-1])) or 0

    monkeypatch.setattr(api, "LIB", Lib())
    monkeypatch.setattr(api, "_raw_stream", lambda i: 100 + i)
    monkeypatch.setattr(api, "_current_device", lambda: current[0])
    monkeypatch.setattr(torch.cuda, "device", device)
    return types.SimpleNamespace(ep=ep, calls=calls, current=current)


def new(cls, dtype, *shape):
    return torch.zeros(shape, dtype=dtype).as_subclass(cls)


def calls_of(ep, cls, odd=None):
    """Every wrapper on tensors of cls; the last operand of each of class odd where it is given."""
    i32, f32, b16, u8 = torch.int32, torch.float32, torch.bfloat16, torch.uint8
    n = lambda dtype, *shape: new(cls, dtype, *shape)
    o = lambda dtype, *shape: new(odd or cls, dtype, *shape)
    lay = lambda: (n(i32, T, K), E, n(i32, E), n(i32, E + 1), n(i32, T, K))
    yield "ep_dispatch_layout", lambda: ep.ep_dispatch_layout(*lay(), o(i32, T * K))
    yield "ep_dispatch_layout_padded", lambda: ep.ep_dispatch_layout_padded(n(i32, T, K), E, CAP, n(i32, E), n(i32, T, K), o(i32, E * CAP))
    R = T * K
    for fmt, x, s in ((ep.EP_RECV_FP8_E4M3_G128, (u8, R, H), (f32, R, 1)), (ep.EP_RECV_BF16, (b16, R, H), None),
                      (ep.EP_RECV_MXFP4_G32, (u8, R, H // 2), (u8, R, H // 32))):
        scale = lambda s=s: n(*s) if s else None
        yield "ep_dispatch", lambda fmt=fmt, x=x, scale=scale: ep.ep_dispatch(n(b16, T, H), n(i32, T, K), n(f32, T, K), fmt, n(*x), scale(), o(f32, R))
        one = lambda x, scale: (n(i32, E), n(i32, E + 1), n(i32, T, K), n(i32, R), n(*x), scale(), o(f32, R))
        yield "ep_layout_dispatch", lambda fmt=fmt, x=x, scale=scale: ep.ep_layout_dispatch(n(i32, T, K), n(b16, T, H), n(f32, T, K), E, 0, fmt, *one(x, scale))
        yield "ep_layout_dispatch_noalloc", lambda fmt=fmt, x=x, scale=scale: ep.ep_layout_dispatch_noalloc(n(i32, T, K), n(b16, T, H), n(f32, T, K), E, 0, fmt, *one(x, scale))
    yield "ep_combine", lambda: ep.ep_combine(n(b16, R, H), n(i32, T, K), n(f32, T, K), o(b16, T, H))
    yield "ep_dispatch_backward", lambda: ep.ep_dispatch_backward(n(b16, R, H), n(i32, T, K), o(b16, T, H))
    yield "ep_combine_backward", lambda: ep.ep_combine_backward(n(b16, T, H), n(b16, R, H), n(i32, T, K), n(f32, T, K), n(b16, R, H), o(f32, T, K))


def operator_calls(ep, cls, odd=None):
    i32, f32, b16, u8 = torch.int32, torch.float32, torch.bfloat16, torch.uint8
    n = lambda dtype, *shape: new(cls, dtype, *shape)
    o = lambda dtype, *shape: new(odd or cls, dtype, *shape)
    yield "ep_route", lambda: ep.ep_route(n(f32, T, E), None, 1, 1, 1, True, 1.0, n(i32, T, K), o(f32, T, K))
    yield "ep_route_backward", lambda: ep.ep_route_backward(n(f32, T, K), n(f32, T, E), n(i32, T, K), 1, True, 1.0, o(f32, T, E))
    yield "ep_quantize_rows", lambda: ep.ep_quantize_rows(n(b16, T, H), ep.EP_RECV_MXFP4_G32, n(u8, T, H // 2), o(u8, T, H // 32))
    yield "ep_dequantize_rows", lambda: ep.ep_dequantize_rows(n(u8, T, H // 2), n(u8, T, H // 32), ep.EP_RECV_MXFP4_G32, o(b16, T, H))
    yield "ep_expert_product", lambda: ep.ep_expert_product(n(u8, T, H // 2), n(u8, T, H // 32), ep.EP_RECV_MXFP4_G32, n(u8, E, 16, H // 2),
                                                            n(u8, E, 16, H // 32), n(i32, E + 1), 0, ep.EP_ACT_NONE, o(b16, T, 16))


@pytest.mark.parametrize("current", [0, 1])
@pytest.mark.parametrize("cls", [OnGpu, OnGpu1])
def test_launched_on_the_operands_device(ep, cls, current):
    """Whatever the receive format, and with that device's stream."""
    ep.current[0] = current
    for make in (calls_of, operator_calls):
        for name, call in make(ep.ep, cls):
            ep.calls.clear()
            call()
            assert ep.calls == [(name, cls.index, 100 + cls.index)]
            assert ep.current[0] == current


@pytest.mark.parametrize("current", [0, 1])
def test_operands_on_several_devices(ep, current):
    """Rows in a peer's memory are launched from the current device, in every
    format; routing, rows and products refuse them."""
    ep.current[0] = current
    for name, call in calls_of(ep.ep, OnGpu, OnGpu1):
        ep.calls.clear()
        call()
        assert ep.calls == [(name, current, 100 + current)]
    for name, call in operator_calls(ep.ep, OnGpu, OnGpu1):
        ep.calls.clear()
        with pytest.raises(ValueError, match="different devices"):
            call()
        assert not ep.calls
