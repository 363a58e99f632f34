"""Python face of the C ABI: the same three calls, taking torch tensors.

Each ``ep_*`` function checks dtypes, devices, shapes and contiguity (the C
side trusts buffer sizes), then passes raw device pointers and the current
HIP stream of the operands' device to libep.so.  Every step of the
computation runs in the library's kernels; torch only owns the memory and the
stream.

``dispatch`` / ``combine`` mirror the pages' call shape
``dispatch(x, topk_idx, topk_weights, num_experts)`` returning received rows
and a handle, and ``combine(...)`` reducing back ([P4] "使用示例 › MoE 训练中
的应用"; [P5] "典型工作流程").
"""

import os
from collections import namedtuple

import torch

from ._lib import (EP_ACT_NONE, EP_ACT_SWIGLU, EP_DTYPE_BF16, EP_DTYPE_F32, EP_MAX_EXPERTS, EP_MAX_TOPK,
                   EP_RECV_BF16, EP_RECV_FP8_E4M3_G128, EP_RECV_MXFP4_G32, EP_SCORE_SIGMOID, LIB, check)

Handle = namedtuple("Handle", "tokens_per_expert expert_offset slot src_token num_experts")
# low-latency (padded) handle: expert e owns rows e*capacity .. e*capacity+capacity-1
PaddedHandle = namedtuple("PaddedHandle", "recv_expert_count slot src_token num_experts capacity")


# without a Stream object, and without the check that the GPU is initialised
# (the operands lie on it): a few us less per call
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _stream(stream):
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(_current_device())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


# EP_DEBUG_CHECK=1: reject expert ids outside [-1, E) before launching.  The
# kernels mask every id outside [0, E), so such ids are legal; an id other
# than -1 out there is usually a caller bug.  The check reads the ids'
# range back to the host (a synchronisation), so it is off by default.
DEBUG_CHECK = os.environ.get("EP_DEBUG_CHECK") == "1"


def _debug_check_ids(topk_idx, num_experts):
    if not DEBUG_CHECK or topk_idx.numel() == 0:
        return
    lo, hi = int(topk_idx.min()), int(topk_idx.max())
    if lo < -1 or hi >= num_experts:
        raise ValueError("EP_DEBUG_CHECK: topk_idx holds ids in [%d, %d], outside [-1, %d)" % (lo, hi, num_experts))


def _need(t, name, dtypes, shape=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.dtype not in dtypes:
        raise TypeError("%s has dtype %s, expected one of %s" % (name, t.dtype, dtypes))
    if not t.is_cuda:  # (a ROCm device tensor reports is_cuda; cheaper than t.device.type)
        raise ValueError("%s must be on a GPU device" % name)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if shape is not None and t.shape != tuple(shape):
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))


_I32 = (torch.int32,)
_IDX = (torch.int32, torch.int64)  # expert ids: int32, or int64 as routers produce them
_F32 = (torch.float32,)
_BF16 = (torch.bfloat16, torch.int16, torch.uint16)
_U8 = (torch.uint8, torch.float8_e4m3fn)
_BYTES = (torch.uint8,)


def _need_recv(format, recv_x, recv_scale, R, H, names=("recv_x", "recv_scale")):
    """Shapes and types of R rows of H channels in a receive format."""
    if format == EP_RECV_FP8_E4M3_G128:
        if H % 128:
            raise ValueError("FP8 dispatch needs hidden % 128 == 0")
        _need(recv_x, names[0], _U8, (R, H))
        _need(recv_scale, names[1], _F32, (R, H // 128))
    elif format == EP_RECV_MXFP4_G32:
        if H % 32:
            raise ValueError("MXFP4 rows need hidden % 32 == 0")
        _need(recv_x, names[0], _BYTES, (R, H // 2))
        _need(recv_scale, names[1], _BYTES, (R, H // 32))
    elif format == EP_RECV_BF16:
        _need(recv_x, names[0], _BF16, (R, H))
    else:
        raise ValueError("unknown receive format %r" % (format,))


def _new_recv(format, R, H, dev):
    """Receive buffers of R rows: (recv_x, recv_scale or None)."""
    if format == EP_RECV_FP8_E4M3_G128:
        return (torch.empty((R, H), dtype=torch.uint8, device=dev),
                torch.empty((R, H // 128), dtype=torch.float32, device=dev))
    if format == EP_RECV_MXFP4_G32:
        return (torch.empty((R, H // 2), dtype=torch.uint8, device=dev),
                torch.empty((R, H // 32), dtype=torch.uint8, device=dev))
    if format == EP_RECV_BF16:
        return torch.empty((R, H), dtype=torch.bfloat16, device=dev), None
    raise ValueError("unknown receive format %r" % (format,))


def _format(fp8, format):
    """The receive format: ``format`` where it is given, else by the fp8 flag."""
    if format is not None:
        return int(format)
    return EP_RECV_FP8_E4M3_G128 if fp8 else EP_RECV_BF16


class _Here:
    """Leaves the current device as it is."""
    __slots__ = ()

    def __enter__(self):
        pass

    def __exit__(self, kind, value, trace):
        pass


_here = _Here()


def _device_of(first, *others):
    """A context with the operands' one device current: launches go to that
    device, and to its current stream."""
    i = first.get_device()
    for t in others:
        if t is not None and t.get_device() != i:
            raise ValueError("operands on different devices: %s and %s" % (first.device, t.device))
    return _here if i == _current_device() else torch.cuda.device(i)


def _transport_device(first, *others):
    """_device_of for layouts, dispatch and combine, whose rows may lie in a
    peer's memory: operands on several devices are launched from the current
    one."""
    i = first.get_device()
    for t in others:
        if t is not None and t.get_device() != i:
            return _here
    return _here if i == _current_device() else torch.cuda.device(i)


def _ids_fn(name, topk_idx):
    """The C entry point for these ids: NAME, or NAME_i64 for int64 ids."""
    return getattr(LIB, name + "_i64") if topk_idx.dtype == torch.int64 else getattr(LIB, name)


def _as_ids(topk_idx):
    """int32 and int64 ids go to the library as they are; other integer
    types are widened to int32."""
    if topk_idx.dtype not in _IDX:
        topk_idx = topk_idx.to(torch.int32)
    return topk_idx.contiguous()


def ep_layout_workspace_bytes(num_tokens, top_k, num_experts):
    """Bytes of device workspace the layout calls need for this shape (0 up
    to 65536 entries, T*K)."""
    return int(LIB.ep_layout_workspace_bytes(int(num_tokens), int(top_k), int(num_experts)))


def ep_dispatch_layout(topk_idx, num_experts, tokens_per_expert, expert_offset, slot, src_token,
                       workspace=None, stream=None):
    """Routing layout into caller-owned int32 tensors: tokens_per_expert [E],
    expert_offset [E+1] (exclusive scan), slot [T, K] (receive row of entry
    (t, k), -1 if masked), src_token [T*K] (token of each row, -1 past
    expert_offset[E]).  Rows of one expert are in ascending token order.
    workspace: uint8/int32 device tensor of ep_layout_workspace_bytes bytes
    (only needed past 65536 entries)."""
    _need(topk_idx, "topk_idx", _IDX)
    _debug_check_ids(topk_idx, num_experts)
    if topk_idx.dim() != 2:
        raise ValueError("topk_idx must be [T, K]")
    T, K = topk_idx.shape
    E = int(num_experts)
    _need(tokens_per_expert, "tokens_per_expert", _I32, (E,))
    _need(expert_offset, "expert_offset", _I32, (E + 1,))
    _need(slot, "slot", _I32, (T, K))
    _need(src_token, "src_token", _I32, (T * K,))
    ws_ptr, ws_bytes = None, 0
    if workspace is not None:
        _need(workspace, "workspace", (torch.uint8, torch.int32))
        ws_ptr, ws_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    with _transport_device(topk_idx, tokens_per_expert, expert_offset, slot, src_token, workspace):
        check("ep_dispatch_layout", _ids_fn("ep_dispatch_layout", topk_idx)(
            topk_idx.data_ptr(), T, K, E, tokens_per_expert.data_ptr(), expert_offset.data_ptr(),
            slot.data_ptr(), src_token.data_ptr(), ws_ptr, ws_bytes, _stream(stream)))


def ep_dispatch_layout_padded(topk_idx, num_experts, capacity, recv_expert_count, slot, src_token,
                              workspace=None, stream=None):
    """Low-latency layout: expert e owns rows e*capacity .. e*capacity +
    capacity - 1; recv_expert_count [E] = min(count, capacity), slot [T, K]
    (-1 for masked or dropped entries), src_token [E*capacity] (unused rows
    are not written)."""
    _need(topk_idx, "topk_idx", _IDX)
    _debug_check_ids(topk_idx, num_experts)
    if topk_idx.dim() != 2:
        raise ValueError("topk_idx must be [T, K]")
    T, K = topk_idx.shape
    E, cap = int(num_experts), int(capacity)
    _need(recv_expert_count, "recv_expert_count", _I32, (E,))
    _need(slot, "slot", _I32, (T, K))
    _need(src_token, "src_token", _I32, (E * cap,))
    ws_ptr, ws_bytes = None, 0
    if workspace is not None:
        _need(workspace, "workspace", (torch.uint8, torch.int32))
        ws_ptr, ws_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    with _transport_device(topk_idx, recv_expert_count, slot, src_token, workspace):
        check("ep_dispatch_layout_padded", _ids_fn("ep_dispatch_layout_padded", topk_idx)(
            topk_idx.data_ptr(), T, K, E, cap, recv_expert_count.data_ptr(), slot.data_ptr(), src_token.data_ptr(),
            ws_ptr, ws_bytes, _stream(stream)))


def ep_dispatch(x, slot, topk_weights, format, recv_x, recv_scale=None, recv_weight=None, stream=None,
                num_rows=None):
    """Copy every token x [T, H] (bf16) into its K receive rows given by slot:
    EP_RECV_FP8_E4M3_G128 writes E4M3FN codes to recv_x (uint8 [rows, H])
    and one float32 scale per 128 channels to recv_scale [rows, H/128];
    EP_RECV_MXFP4_G32 writes E2M1 codes (uint8 [rows, H/2], the even channel
    in the low half) and one scale byte per 32 channels (uint8 [rows, H/32]);
    EP_RECV_BF16 copies the bf16 bits to recv_x (bf16 [rows, H]).
    recv_weight [rows] (optional) receives topk_weights[t, k].  num_rows:
    rows of the receive buffers (T*K by default; E*capacity for a padded
    slot)."""
    _need(x, "x", _BF16)
    if x.dim() != 2:
        raise ValueError("x must be [T, H]")
    T, H = x.shape
    _need(slot, "slot", _I32)
    if slot.dim() != 2 or slot.shape[0] != T:
        raise ValueError("slot must be [T, K]")
    K = slot.shape[1]
    R = T * K if num_rows is None else int(num_rows)
    if topk_weights is not None:
        _need(topk_weights, "topk_weights", _F32, (T, K))
    _need_recv(format, recv_x, recv_scale, R, H)
    if recv_weight is not None:
        _need(recv_weight, "recv_weight", _F32, (R,))
    with _transport_device(x, slot, topk_weights, recv_x, recv_scale, recv_weight):
        check("ep_dispatch", LIB.ep_dispatch(
            x.data_ptr(), T, H, K, slot.data_ptr(),
            topk_weights.data_ptr() if topk_weights is not None else None, int(format), recv_x.data_ptr(),
            recv_scale.data_ptr() if recv_scale is not None else None,
            recv_weight.data_ptr() if recv_weight is not None else None, _stream(stream)))


def _check_layout_dispatch(topk_idx, x, topk_weights, num_experts, capacity, format, tokens_per_expert,
                           expert_offset, slot, src_token, recv_x, recv_scale, recv_weight):
    """Shape and dtype checks of ep_layout_dispatch's tensors; returns T, H, K."""
    _need(topk_idx, "topk_idx", _IDX)
    _debug_check_ids(topk_idx, num_experts)
    if topk_idx.dim() != 2:
        raise ValueError("topk_idx must be [T, K]")
    T, K = topk_idx.shape
    E, cap = int(num_experts), int(capacity)
    if cap < 0:
        raise ValueError("capacity must be >= 0")
    R = E * cap if cap else T * K
    _need(x, "x", _BF16)
    if x.dim() != 2 or x.shape[0] != T:
        raise ValueError("x must be [T, H]")
    H = x.shape[1]
    _need(tokens_per_expert, "tokens_per_expert", _I32, (E,))
    if cap == 0:
        _need(expert_offset, "expert_offset", _I32, (E + 1,))
    elif expert_offset is not None:
        raise ValueError("expert_offset is not used by the padded layout; pass None")
    _need(slot, "slot", _I32, (T, K))
    _need(src_token, "src_token", _I32, (R,))
    if topk_weights is not None:
        _need(topk_weights, "topk_weights", _F32, (T, K))
    _need_recv(format, recv_x, recv_scale, R, H)
    if recv_weight is not None:
        _need(recv_weight, "recv_weight", _F32, (R,))
    return T, H, K


def ep_layout_dispatch(topk_idx, x, topk_weights, num_experts, capacity, format, tokens_per_expert,
                       expert_offset, slot, src_token, recv_x, recv_scale=None, recv_weight=None, workspace=None,
                       stream=None):
    """Layout and dispatch in one call (one launch up to 65536 entries).
    capacity 0: packed layout (expert_offset [E+1], src_token [T*K], T*K
    receive rows); capacity > 0: padded layout (expert_offset None,
    src_token [E*capacity], E*capacity receive rows)."""
    T, H, K = _check_layout_dispatch(topk_idx, x, topk_weights, num_experts, capacity, format, tokens_per_expert,
                                     expert_offset, slot, src_token, recv_x, recv_scale, recv_weight)
    E, cap = int(num_experts), int(capacity)
    ws_ptr, ws_bytes = None, 0
    if workspace is not None:
        _need(workspace, "workspace", (torch.uint8, torch.int32))
        ws_ptr, ws_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    with _transport_device(x, topk_idx, topk_weights, tokens_per_expert, expert_offset, slot, src_token,
                           recv_x, recv_scale, recv_weight, workspace):
        check("ep_layout_dispatch", _ids_fn("ep_layout_dispatch", topk_idx)(
            topk_idx.data_ptr(), x.data_ptr(), topk_weights.data_ptr() if topk_weights is not None else None, T, H, K,
            E, cap, int(format), tokens_per_expert.data_ptr(),
            expert_offset.data_ptr() if expert_offset is not None else None, slot.data_ptr(), src_token.data_ptr(),
            recv_x.data_ptr(), recv_scale.data_ptr() if recv_scale is not None else None,
            recv_weight.data_ptr() if recv_weight is not None else None, ws_ptr, ws_bytes, _stream(stream)))


def ep_layout_dispatch_noalloc(topk_idx, x, topk_weights, num_experts, capacity, format, tokens_per_expert,
                               expert_offset, slot, src_token, recv_x, recv_scale=None, recv_weight=None,
                               stream=None):
    """ep_layout_dispatch without a workspace: the library's own per-GPU
    scratch (EP_NOALLOC_SCRATCH_BYTES) holds the layout's histograms, so the
    call allocates nothing.  int32 ids only.  Calls that overlap on one GPU
    race on that scratch; issue them on one stream."""
    if topk_idx.dtype != torch.int32:
        raise TypeError("ep_layout_dispatch_noalloc takes int32 topk_idx")
    T, H, K = _check_layout_dispatch(topk_idx, x, topk_weights, num_experts, capacity, format, tokens_per_expert,
                                     expert_offset, slot, src_token, recv_x, recv_scale, recv_weight)
    with _transport_device(x, topk_idx, topk_weights, tokens_per_expert, expert_offset, slot, src_token,
                           recv_x, recv_scale, recv_weight):
        check("ep_layout_dispatch_noalloc", LIB.ep_layout_dispatch_noalloc(
            topk_idx.data_ptr(), x.data_ptr(), topk_weights.data_ptr() if topk_weights is not None else None, T, H, K,
            int(num_experts), int(capacity), int(format), tokens_per_expert.data_ptr(),
            expert_offset.data_ptr() if expert_offset is not None else None, slot.data_ptr(), src_token.data_ptr(),
            recv_x.data_ptr(), recv_scale.data_ptr() if recv_scale is not None else None,
            recv_weight.data_ptr() if recv_weight is not None else None, _stream(stream)))


def ep_combine(y, slot, topk_weights, out, stream=None, num_rows=None):
    """out[t] = BF16(sum over k of topk_weights[t, k] * y[slot[t, k]]), in
    binary32, ascending k, each product rounded before it is added.
    y: bf16 [rows, H] in receive order; out: bf16 [T, H].  num_rows: rows
    of y (T*K by default; E*capacity for a padded slot)."""
    _need(slot, "slot", _I32)
    if slot.dim() != 2:
        raise ValueError("slot must be [T, K]")
    T, K = slot.shape
    _need(y, "y", _BF16)
    R = T * K if num_rows is None else int(num_rows)
    if y.dim() != 2 or y.shape[0] != R:
        raise ValueError("y must be [%d, H]" % R)
    H = y.shape[1]
    _need(topk_weights, "topk_weights", _F32, (T, K))
    _need(out, "out", _BF16, (T, H))
    with _transport_device(y, slot, topk_weights, out):
        check("ep_combine", LIB.ep_combine(y.data_ptr(), slot.data_ptr(), topk_weights.data_ptr(), T, H, K,
                                           out.data_ptr(), _stream(stream)))


def ep_dispatch_backward(grad_recv, slot, grad_x, stream=None, num_rows=None):
    """grad_x [T, H] = sum over k of grad_recv[slot[t, k]] (bf16)."""
    _need(slot, "slot", _I32)
    if slot.dim() != 2:
        raise ValueError("slot must be [T, K]")
    T, K = slot.shape
    _need(grad_recv, "grad_recv", _BF16)
    R = T * K if num_rows is None else int(num_rows)
    if grad_recv.dim() != 2 or grad_recv.shape[0] != R:
        raise ValueError("grad_recv must be [%d, H]" % R)
    H = grad_recv.shape[1]
    _need(grad_x, "grad_x", _BF16, (T, H))
    with _transport_device(grad_recv, slot, grad_x):
        check("ep_dispatch_backward", LIB.ep_dispatch_backward(grad_recv.data_ptr(), slot.data_ptr(), T, H, K,
                                                               grad_x.data_ptr(), _stream(stream)))


def ep_combine_backward(grad_out, y, slot, topk_weights, grad_y, grad_w=None, stream=None, num_rows=None):
    """grad_y rows = w * grad_out (bf16); grad_w [T, K] = row dot products
    (float32), or skipped when grad_w is None (y may then be None)."""
    _need(slot, "slot", _I32)
    if slot.dim() != 2:
        raise ValueError("slot must be [T, K]")
    T, K = slot.shape
    _need(grad_out, "grad_out", _BF16)
    if grad_out.dim() != 2 or grad_out.shape[0] != T:
        raise ValueError("grad_out must be [T, H]")
    H = grad_out.shape[1]
    R = T * K if num_rows is None else int(num_rows)
    _need(topk_weights, "topk_weights", _F32, (T, K))
    _need(grad_y, "grad_y", _BF16, (R, H))
    if grad_w is not None:
        _need(y, "y", _BF16, (R, H))
        _need(grad_w, "grad_w", _F32, (T, K))
    with _transport_device(grad_out, y if grad_w is not None else None, slot, topk_weights, grad_y, grad_w):
        check("ep_combine_backward", LIB.ep_combine_backward(
            grad_out.data_ptr(), y.data_ptr() if y is not None else None, slot.data_ptr(), topk_weights.data_ptr(),
            T, H, K, grad_y.data_ptr(), grad_w.data_ptr() if grad_w is not None else None, _stream(stream)))


def _logits_dtype(logits):
    return EP_DTYPE_BF16 if logits.dtype == torch.bfloat16 else EP_DTYPE_F32


_LOGITS = (torch.float32, torch.bfloat16)


def ep_route(logits, bias, n_group, topk_group, score, renormalize, scale, topk_idx, topk_weights, stream=None):
    """Router logits [T, E] (float32 or bf16) to topk_idx (int32 [T, K], by
    descending score, -1 where no expert is left) and topk_weights (float32
    [T, K]).  score: EP_SCORE_SIGMOID or EP_SCORE_SOFTMAX; bias (float32 [E]
    or None) is added to the scores for the choice only; the topk_group best
    of n_group groups are kept; renormalize divides by the sum of the chosen
    scores; scale multiplies the weights."""
    _need(logits, "logits", _LOGITS)
    if logits.dim() != 2:
        raise ValueError("logits must be [T, E]")
    T, E = logits.shape
    if bias is not None:
        _need(bias, "bias", _F32, (E,))
    _need(topk_idx, "topk_idx", _I32)
    if topk_idx.dim() != 2 or topk_idx.shape[0] != T:
        raise ValueError("topk_idx must be [T, K]")
    K = topk_idx.shape[1]
    _need(topk_weights, "topk_weights", _F32, (T, K))
    with _device_of(logits, bias, topk_idx, topk_weights):
        check("ep_route", LIB.ep_route(
            logits.data_ptr(), _logits_dtype(logits), bias.data_ptr() if bias is not None else None, T, E, K,
            int(n_group), int(topk_group), int(score), int(bool(renormalize)), float(scale), topk_idx.data_ptr(),
            topk_weights.data_ptr(), _stream(stream)))


def ep_route_backward(grad_w, logits, topk_idx, score, renormalize, scale, grad_logits, stream=None):
    """Gradient of ep_route's weights: grad_w float32 [T, K] to grad_logits
    [T, E], of the logits' type.  Entries of topk_idx outside [0, E) count
    for nothing."""
    _need(logits, "logits", _LOGITS)
    if logits.dim() != 2:
        raise ValueError("logits must be [T, E]")
    T, E = logits.shape
    _need(topk_idx, "topk_idx", _I32)
    if topk_idx.dim() != 2 or topk_idx.shape[0] != T:
        raise ValueError("topk_idx must be [T, K]")
    K = topk_idx.shape[1]
    _need(grad_w, "grad_w", _F32, (T, K))
    _need(grad_logits, "grad_logits", (logits.dtype,), (T, E))
    with _device_of(logits, grad_w, topk_idx, grad_logits):
        check("ep_route_backward", LIB.ep_route_backward(
            grad_w.data_ptr(), logits.data_ptr(), _logits_dtype(logits), topk_idx.data_ptr(), T, E, K, int(score),
            int(bool(renormalize)), float(scale), grad_logits.data_ptr(), _stream(stream)))


def ep_quantize_rows(x, format, q, scale, stream=None):
    """Rows x [R, H] (bf16) to the codes and scales dispatch would write for
    them: FP8 (uint8 [R, H], float32 [R, H/128]) or MXFP4 (uint8 [R, H/2],
    uint8 [R, H/32])."""
    _need(x, "x", _BF16)
    if x.dim() != 2:
        raise ValueError("x must be [R, H]")
    R, H = x.shape
    if format not in (EP_RECV_FP8_E4M3_G128, EP_RECV_MXFP4_G32):
        raise ValueError("rows are quantised to FP8 or MXFP4, not format %r" % (format,))
    _need_recv(format, q, scale, R, H, ("q", "scale"))
    with _device_of(x, q, scale):
        check("ep_quantize_rows", LIB.ep_quantize_rows(x.data_ptr(), R, H, int(format), q.data_ptr(),
                                                       scale.data_ptr(), _stream(stream)))


def ep_dequantize_rows(q, scale, format, x, stream=None):
    """The values (bf16 [R, H]) that FP8 or MXFP4 codes and scales stand for."""
    _need(x, "x", _BF16)
    if x.dim() != 2:
        raise ValueError("x must be [R, H]")
    R, H = x.shape
    if format not in (EP_RECV_FP8_E4M3_G128, EP_RECV_MXFP4_G32):
        raise ValueError("rows are dequantised from FP8 or MXFP4, not format %r" % (format,))
    _need_recv(format, q, scale, R, H, ("q", "scale"))
    with _device_of(x, q, scale):
        check("ep_dequantize_rows", LIB.ep_dequantize_rows(q.data_ptr(), scale.data_ptr(), R, H, int(format),
                                                           x.data_ptr(), _stream(stream)))


def ep_expert_product(a, a_scale, format, w, w_scale, expert_rows, capacity, activation, y, stream=None):
    """y[r] = act(w[e(r)] @ a[r]) for every expert's rows.  a, a_scale: rows in
    MXFP4 or FP8 (format EP_RECV_*); w uint8 [E, N, H/2] and w_scale uint8
    [E, N, H/32]: MXFP4; expert_rows: expert_offset int32 [E+1] (capacity 0)
    or recv_expert_count int32 [E] (capacity > 0, rows = E*capacity);
    activation EP_ACT_NONE (y bf16 [rows, N]) or EP_ACT_SWIGLU (y bf16 [rows,
    N/2]: silu of the first N/2 products times the others).  Rows of no
    expert are left untouched."""
    _need(w, "w", _BYTES)
    if w.dim() != 3:
        raise ValueError("w must be [E, N, H/2]")
    E, N, H = w.shape[0], w.shape[1], w.shape[2] * 2
    if H % 128:
        raise ValueError("the product needs hidden % 128 == 0")
    _need(w_scale, "w_scale", _BYTES, (E, N, H // 32))
    if format not in (EP_RECV_FP8_E4M3_G128, EP_RECV_MXFP4_G32):
        raise ValueError("the product takes FP8 or MXFP4 rows, not format %r" % (format,))
    if not isinstance(a, torch.Tensor) or a.dim() != 2:
        raise ValueError("a must be [rows, bytes of a row]")
    R, cap = a.shape[0], int(capacity)
    _need_recv(format, a, a_scale, R, H, ("a", "a_scale"))
    if cap < 0 or (cap > 0 and R != E * cap):
        raise ValueError("capacity %d does not fit %d rows of %d experts" % (cap, R, E))
    _need(expert_rows, "expert_rows", _I32, (E,) if cap else (E + 1,))
    if activation not in (EP_ACT_NONE, EP_ACT_SWIGLU):
        raise ValueError("unknown activation %r" % (activation,))
    if N % (16 if activation == EP_ACT_SWIGLU else 8):
        raise ValueError("the product needs out channels in multiples of 8")
    _need(y, "y", _BF16, (R, N // 2 if activation == EP_ACT_SWIGLU else N))
    with _device_of(a, a_scale, w, w_scale, expert_rows, y):
        check("ep_expert_product", LIB.ep_expert_product(
            a.data_ptr(), a_scale.data_ptr(), int(format), w.data_ptr(), w_scale.data_ptr(), expert_rows.data_ptr(),
            R, E, cap, H, N, int(activation), y.data_ptr(), _stream(stream)))


def _rows_shape(expert_rows, E, R, capacity):
    """Checks of an expert layer's rows; the address of expert_rows, or None."""
    if capacity < 0 or (capacity > 0 and R != E * capacity):
        raise ValueError("capacity %d does not fit %d rows of %d experts" % (capacity, R, E))
    if expert_rows is None:
        if E != 1 or capacity != 0:
            raise ValueError("without expert_rows there is one matrix and no capacity")
        return None
    _need(expert_rows, "expert_rows", _I32, (E,) if capacity else (E + 1,))
    return expert_rows.data_ptr()


def ep_expert_linear(a, w, expert_rows, capacity, activation, y, bias=None, residual=None, p=None, stream=None):
    """y[r] = act(w[e(r)] @ a[r] + bias[e(r)]) + residual[r] in bf16.  a [rows,
    H]; w [E, N, H]; bias [E, N] or None; expert_rows: as ep_expert_product's,
    or None (E 1, capacity 0) where every row is the one matrix's; activation
    EP_ACT_NONE (y [rows, N]) or EP_ACT_SWIGLU (y [rows, N/2]); residual of
    y's shape or None, may be y itself; p [rows, N] or None (EP_ACT_SWIGLU)
    receives the rows before the activation.  Rows of no expert are left
    untouched."""
    _need(w, "w", _BF16)
    if w.dim() != 3:
        raise ValueError("w must be [E, N, H]")
    E, N, H = w.shape
    if activation not in (EP_ACT_NONE, EP_ACT_SWIGLU):
        raise ValueError("unknown activation %r" % (activation,))
    gated = activation == EP_ACT_SWIGLU
    if H % 8 or N % (16 if gated else 8):
        raise ValueError("the layer needs hidden and out channels in multiples of 8, gate and up each")
    _need(a, "a", _BF16)
    if a.dim() != 2 or a.shape[1] != H:
        raise ValueError("a must be [rows, %d]" % H)
    R, cap = a.shape[0], int(capacity)
    rows = _rows_shape(expert_rows, E, R, cap)
    out = N // 2 if gated else N
    _need(y, "y", _BF16, (R, out))
    if bias is not None:
        _need(bias, "bias", _BF16, (E, N))
    if residual is not None:
        _need(residual, "residual", _BF16, (R, out))
    if p is not None:
        if not gated:
            raise ValueError("p belongs to a gated layer")
        _need(p, "p", _BF16, (R, N))
    with _device_of(a, w, expert_rows, bias, residual, p, y):
        check("ep_expert_linear", LIB.ep_expert_linear(
            a.data_ptr(), w.data_ptr(), bias.data_ptr() if bias is not None else None,
            residual.data_ptr() if residual is not None else None, rows, R, E, cap, H, N, int(activation),
            p.data_ptr() if p is not None else None, y.data_ptr(), _stream(stream)))


def ep_expert_linear_backward(grad_y, w, expert_rows, capacity, grad_a, p=None, stream=None):
    """Gradient of ep_expert_linear w.r.t. its rows: grad_y [rows, N] and w
    [E, N, H] to grad_a [rows, H]; with p [rows, 2H], what the gated layer
    before it kept, on to the gradient of p, grad_a [rows, 2H] (may be p
    itself)."""
    _need(w, "w", _BF16)
    if w.dim() != 3:
        raise ValueError("w must be [E, N, H]")
    E, N, H = w.shape
    if H % 8 or N % 8:
        raise ValueError("the layer needs hidden and out channels in multiples of 8")
    _need(grad_y, "grad_y", _BF16)
    if grad_y.dim() != 2 or grad_y.shape[1] != N:
        raise ValueError("grad_y must be [rows, %d]" % N)
    R, cap = grad_y.shape[0], int(capacity)
    rows = _rows_shape(expert_rows, E, R, cap)
    if p is not None:
        _need(p, "p", _BF16, (R, 2 * H))
    _need(grad_a, "grad_a", _BF16, (R, 2 * H if p is not None else H))
    with _device_of(grad_y, w, expert_rows, p, grad_a):
        check("ep_expert_linear_backward", LIB.ep_expert_linear_backward(
            grad_y.data_ptr(), w.data_ptr(), p.data_ptr() if p is not None else None, rows, R, E, cap, H, N,
            grad_a.data_ptr(), _stream(stream)))


def ep_expert_linear_backward_weights(grad_y, a, expert_rows, capacity, grad_w, grad_bias=None, accumulate=False,
                                      stream=None):
    """Gradients of ep_expert_linear w.r.t. its weights and biases: grad_y
    [rows, N] and a [rows, H] (bf16) to grad_w [E, N, H] (float32 or bf16) and
    grad_bias [E, N] (of the same type) or None; accumulate adds to what is
    there.  Experts without rows get zeros."""
    _need(grad_w, "grad_w", (torch.float32, torch.bfloat16))
    if grad_w.dim() != 3:
        raise ValueError("grad_w must be [E, N, H]")
    E, N, H = grad_w.shape
    if H % 8 or N % 8:
        raise ValueError("the layer needs hidden and out channels in multiples of 8")
    _need(grad_y, "grad_y", _BF16)
    if grad_y.dim() != 2 or grad_y.shape[1] != N:
        raise ValueError("grad_y must be [rows, %d]" % N)
    R, cap = grad_y.shape[0], int(capacity)
    _need(a, "a", _BF16, (R, H))
    rows = _rows_shape(expert_rows, E, R, cap)
    if grad_bias is not None:
        _need(grad_bias, "grad_bias", (grad_w.dtype,), (E, N))
    with _device_of(grad_y, a, expert_rows, grad_w, grad_bias):
        check("ep_expert_linear_backward_weights", LIB.ep_expert_linear_backward_weights(
            grad_y.data_ptr(), a.data_ptr(), rows, R, E, cap, H, N, _logits_dtype(grad_w), int(bool(accumulate)),
            grad_w.data_ptr(), grad_bias.data_ptr() if grad_bias is not None else None, _stream(stream)))


def ep_cast_fp8_e4m3(inp, out, stream=None):
    """The binary32 -> E4M3FN conversion dispatch uses (round to nearest
    even, saturating at +-448), elementwise: inp float32, out uint8 of the
    same shape."""
    _need(inp, "in", _F32)
    _need(out, "out", _U8, tuple(inp.shape))
    with _device_of(inp, out):
        check("ep_cast_fp8_e4m3", LIB.ep_cast_fp8_e4m3(inp.data_ptr(), out.data_ptr(), inp.numel(),
                                                       _stream(stream)))


# ---- convenience wrappers that allocate their outputs ----------------------

def layout(topk_idx, num_experts, stream=None):
    """Routing layout of ``topk_idx`` [T, K] (int32 or int64) -> Handle."""
    topk_idx = _as_ids(topk_idx)
    T, K = topk_idx.shape
    E = int(num_experts)
    if not 1 <= E <= EP_MAX_EXPERTS or not 1 <= K <= EP_MAX_TOPK:
        raise ValueError("unsupported num_experts=%d / top_k=%d" % (E, K))
    dev = topk_idx.device
    counts = torch.empty(E, dtype=torch.int32, device=dev)
    offsets = torch.empty(E + 1, dtype=torch.int32, device=dev)
    slot = torch.empty((T, K), dtype=torch.int32, device=dev)
    src = torch.empty(T * K, dtype=torch.int32, device=dev)
    nb = ep_layout_workspace_bytes(T, K, E)
    ws = torch.empty(nb, dtype=torch.uint8, device=dev) if nb else None
    ep_dispatch_layout(topk_idx, E, counts, offsets, slot, src, ws, stream)
    return Handle(counts, offsets, slot, src, E)


def dispatch(x, topk_idx, topk_weights, num_experts, fp8=True, handle=None, stream=None, format=None):
    """Permute tokens into expert-major rows.

    Returns (recv_x, recv_scale, recv_weight, handle): recv_x is uint8 E4M3FN
    [T*K, H] with recv_scale float32 [T*K, H/128] when ``fp8``, else bfloat16
    [T*K, H] with recv_scale None; recv_weight float32 [T*K] (None if
    ``topk_weights`` is None).  ``format`` (EP_RECV_*) picks the receive
    format instead of ``fp8``: EP_RECV_MXFP4_G32 gives uint8 [T*K, H/2] codes
    and uint8 [T*K, H/32] scales.  Rows expert_offset[e] .. expert_offset[e+1]-1
    belong to expert e.
    """
    T, H = x.shape
    dev = x.device
    if handle is None:
        topk_idx = _as_ids(topk_idx)
    K = handle.slot.shape[1] if handle is not None else topk_idx.shape[1]
    recv_weight = None
    if topk_weights is not None:
        topk_weights = topk_weights.to(torch.float32).contiguous()
        recv_weight = torch.empty(T * K, dtype=torch.float32, device=dev)
    fmt = _format(fp8, format)
    recv_x, recv_scale = _new_recv(fmt, T * K, H, dev)
    if handle is not None:
        ep_dispatch(x, handle.slot, topk_weights, fmt, recv_x, recv_scale, recv_weight, stream)
        return recv_x, recv_scale, recv_weight, handle
    E = int(num_experts)
    if not 1 <= E <= EP_MAX_EXPERTS or not 1 <= K <= EP_MAX_TOPK:
        raise ValueError("unsupported num_experts=%d / top_k=%d" % (E, K))
    counts = torch.empty(E, dtype=torch.int32, device=dev)
    offsets = torch.empty(E + 1, dtype=torch.int32, device=dev)
    slot = torch.empty((T, K), dtype=torch.int32, device=dev)
    src = torch.empty(T * K, dtype=torch.int32, device=dev)
    nb = ep_layout_workspace_bytes(T, K, E)
    ws = torch.empty(nb, dtype=torch.uint8, device=dev) if nb else None
    ep_layout_dispatch(topk_idx, x, topk_weights, E, 0, fmt, counts, offsets, slot, src, recv_x, recv_scale,
                       recv_weight, ws, stream)
    return recv_x, recv_scale, recv_weight, Handle(counts, offsets, slot, src, E)


def combine(y, handle, topk_weights, stream=None):
    """Weighted reduction of expert outputs ``y`` [T*K, H] (bf16, receive
    order) back to token order -> bfloat16 [T, H]."""
    T = handle.slot.shape[0]
    out = torch.empty((T, y.shape[1]), dtype=torch.bfloat16, device=y.device)
    ep_combine(y, handle.slot, topk_weights.to(torch.float32).contiguous(), out, stream)
    return out


def layout_padded(topk_idx, num_experts, capacity, stream=None):
    """Low-latency layout with ``capacity`` rows per expert -> PaddedHandle."""
    topk_idx = _as_ids(topk_idx)
    T, K = topk_idx.shape
    E, cap = int(num_experts), int(capacity)
    dev = topk_idx.device
    count = torch.empty(E, dtype=torch.int32, device=dev)
    slot = torch.empty((T, K), dtype=torch.int32, device=dev)
    src = torch.empty(E * cap, dtype=torch.int32, device=dev)
    nb = ep_layout_workspace_bytes(T, K, E)
    ws = torch.empty(nb, dtype=torch.uint8, device=dev) if nb else None
    ep_dispatch_layout_padded(topk_idx, E, cap, count, slot, src, ws, stream)
    return PaddedHandle(count, slot, src, E, cap)


def low_latency_dispatch(x, topk_idx, num_max_tokens, num_experts, fp8=True, stream=None, format=None):
    """Decode-time dispatch into a padded buffer, shaped like the pages'
    ``low_latency_dispatch(hidden_states, topk_idx, num_max_tokens,
    num_experts)`` ([P4] "使用示例 › 推理解码阶段的应用").

    Returns (recv_x [E, num_max_tokens, H], recv_scale [E, num_max_tokens,
    H/128] or None, recv_expert_count [E], handle).  ``format`` (EP_RECV_*)
    picks the receive format instead of ``fp8``; MXFP4 rows have H/2 bytes
    and H/32 scale bytes.
    """
    topk_idx = _as_ids(topk_idx)
    T, H = x.shape
    K = topk_idx.shape[1]
    E, cap = int(num_experts), int(num_max_tokens)
    if cap < 1:
        raise ValueError("num_max_tokens must be >= 1")
    dev = x.device
    count = torch.empty(E, dtype=torch.int32, device=dev)
    slot = torch.empty((T, K), dtype=torch.int32, device=dev)
    src = torch.empty(E * cap, dtype=torch.int32, device=dev)
    nb = ep_layout_workspace_bytes(T, K, E)
    ws = torch.empty(nb, dtype=torch.uint8, device=dev) if nb else None
    fmt = _format(fp8, format)
    recv_x, recv_scale = _new_recv(fmt, E * cap, H, dev)
    ep_layout_dispatch(topk_idx, x, None, E, cap, fmt, count, None, slot, src, recv_x, recv_scale, None, ws, stream)
    if recv_scale is not None:
        recv_scale = recv_scale.view(E, cap, -1)
    return recv_x.view(E, cap, -1), recv_scale, count, PaddedHandle(count, slot, src, E, cap)


def low_latency_combine(y, handle, topk_weights, stream=None):
    """Weighted reduction of padded expert outputs y [E, capacity, H] (bf16)
    back to token order -> bfloat16 [T, H]."""
    E, cap = handle.num_experts, handle.capacity
    H = y.shape[-1]
    y2 = y.reshape(E * cap, H)
    T = handle.slot.shape[0]
    out = torch.empty((T, H), dtype=torch.bfloat16, device=y.device)
    ep_combine(y2, handle.slot, topk_weights.to(torch.float32).contiguous(), out, stream, num_rows=E * cap)
    return out


def dispatch_backward(grad_recv, handle, stream=None):
    """Gradient of dispatch w.r.t. x: the K copies' gradients summed -> bf16 [T, H]."""
    T = handle.slot.shape[0]
    R = grad_recv.shape[0]
    out = torch.empty((T, grad_recv.shape[1]), dtype=torch.bfloat16, device=grad_recv.device)
    ep_dispatch_backward(grad_recv, handle.slot, out, stream, num_rows=R)
    return out


def combine_backward(grad_out, y, handle, topk_weights, stream=None):
    """Gradients of combine -> (grad_y bf16 [rows, H], grad_w float32 [T, K]).
    Rows no entry maps to are zero-filled first (a torch fill)."""
    T, K = handle.slot.shape
    R, H = y.shape
    grad_y = torch.zeros((R, H), dtype=torch.bfloat16, device=y.device)
    grad_w = torch.empty((T, K), dtype=torch.float32, device=y.device)
    ep_combine_backward(grad_out, y, handle.slot, topk_weights.to(torch.float32).contiguous(), grad_y, grad_w,
                        stream, num_rows=R)
    return grad_y, grad_w


def route(logits, top_k, bias=None, n_group=1, topk_group=1, score=EP_SCORE_SIGMOID, renormalize=True, scale=1.0,
          stream=None):
    """Router logits [T, E] -> (topk_idx int32 [T, K], topk_weights float32
    [T, K]), as dispatch and combine take them (see ep_route)."""
    T, K = logits.shape[0], int(top_k)
    if not 1 <= K <= EP_MAX_TOPK:
        raise ValueError("unsupported top_k=%d" % K)
    topk_idx = torch.empty((T, K), dtype=torch.int32, device=logits.device)
    topk_weights = torch.empty((T, K), dtype=torch.float32, device=logits.device)
    ep_route(logits, bias, n_group, topk_group, score, renormalize, scale, topk_idx, topk_weights, stream)
    return topk_idx, topk_weights


def route_backward(grad_w, logits, topk_idx, score=EP_SCORE_SIGMOID, renormalize=True, scale=1.0, stream=None):
    """Gradient of route's weights (combine_backward's grad_w) w.r.t. the
    logits -> [T, E] of their type."""
    grad_logits = torch.empty_like(logits)
    ep_route_backward(grad_w, logits, topk_idx, score, renormalize, scale, grad_logits, stream)
    return grad_logits


def quantize_rows(x, format=EP_RECV_MXFP4_G32, stream=None):
    """Rows x [R, H] (bf16) -> (codes, scales), as dispatch leaves them."""
    if format not in (EP_RECV_FP8_E4M3_G128, EP_RECV_MXFP4_G32):
        raise ValueError("rows are quantised to FP8 or MXFP4, not format %r" % (format,))
    q, scale = _new_recv(format, x.shape[0], x.shape[1], x.device)
    ep_quantize_rows(x, format, q, scale, stream)
    return q, scale


def dequantize_rows(q, scale, format=EP_RECV_MXFP4_G32, stream=None):
    """Codes and scales -> the bf16 rows [R, H] they stand for."""
    H = q.shape[1] * (2 if format == EP_RECV_MXFP4_G32 else 1)
    x = torch.empty((q.shape[0], H), dtype=torch.bfloat16, device=q.device)
    ep_dequantize_rows(q, scale, format, x, stream)
    return x


def expert_product(a, a_scale, w, w_scale, handle, activation=EP_ACT_NONE, stream=None):
    """Every expert's product on its rows -> bf16 [rows, N] (N/2 channels with
    EP_ACT_SWIGLU), [E, capacity, ..] for a PaddedHandle.  a, a_scale: as
    dispatch (or low_latency_dispatch) returned them with ``handle``, or
    quantize_rows made them; uint8 scales mean MXFP4 rows, float32 scales
    FP8.  Rows of no expert hold no defined values."""
    format = EP_RECV_MXFP4_G32 if a_scale.dtype == torch.uint8 else EP_RECV_FP8_E4M3_G128
    padded = isinstance(handle, PaddedHandle)
    for name, t in (("a", a), ("a_scale", a_scale), ("w", w)):
        if t.dim() < 2 or not t.is_contiguous():  # (a copy made here would be on the current stream, not on ``stream``)
            raise ValueError("%s must be contiguous rows" % name)
    a2, s2 = a.view(-1, a.shape[-1]), a_scale.view(-1, a_scale.shape[-1])
    out = w.shape[1] // 2 if activation == EP_ACT_SWIGLU else w.shape[1]
    y = torch.empty((a2.shape[0], out), dtype=torch.bfloat16, device=a.device)
    ep_expert_product(a2, s2, format, w, w_scale, handle.recv_expert_count if padded else handle.expert_offset,
                      handle.capacity if padded else 0, activation, y, stream)
    return y.view(handle.num_experts, handle.capacity, out) if padded else y


def _flat(name, t):
    if t.dim() < 2 or not t.is_contiguous():  # (a copy made here would be on the current stream, not on ``stream``)
        raise ValueError("%s must be contiguous rows" % name)
    return t if t.dim() == 2 else t.view(-1, t.shape[-1])  # (a view costs the host a us)


def _expert_rows(handle):
    """expert_rows and capacity of a handle (None: every row is one matrix's)."""
    if handle is None:
        return None, 0
    if isinstance(handle, PaddedHandle):
        return handle.recv_expert_count, handle.capacity
    return handle.expert_offset, 0


def _matrices(w):
    return w.unsqueeze(0) if w.dim() == 2 else w  # (one matrix may come without its expert dimension)


def _as_rows(t, handle):
    return t.view(handle.num_experts, handle.capacity, -1) if isinstance(handle, PaddedHandle) else t


def expert_linear(a, w, handle, bias=None, activation=EP_ACT_NONE, residual=None, save=False, stream=None):
    """Every expert's bf16 layer on its rows -> bf16 [rows, N] (N/2 channels
    with EP_ACT_SWIGLU), [E, capacity, ..] for a PaddedHandle.  a: as dispatch
    (or low_latency_dispatch) returned it with ``handle`` in EP_RECV_BF16; w
    [E, N, H], bias [E, N].  ``handle`` None: one matrix w ([N, H], or [1, N,
    H]; bias [N] or [1, N]) for all rows, a shared expert's.  residual (of the
    result's shape) is added behind the activation.  With save (EP_ACT_SWIGLU)
    -> (y, p), p [rows, N] being what expert_linear_backward needs.  Rows of
    no expert hold no defined values."""
    rows, cap = _expert_rows(handle)
    a2, w = _flat("a", a), _matrices(w)
    if w.dim() != 3:
        raise ValueError("w must be [E, N, H]")
    N = w.shape[1]
    y = torch.empty((a2.shape[0], N // 2 if activation == EP_ACT_SWIGLU else N), dtype=torch.bfloat16, device=a.device)
    p = torch.empty((a2.shape[0], N), dtype=torch.bfloat16, device=a.device) if save else None
    if bias is not None and bias.dim() == 1:
        bias = bias.unsqueeze(0)
    ep_expert_linear(a2, w, rows, cap, activation, y, bias, _flat("residual", residual) if residual is not None else None,
                     p, stream)
    return (_as_rows(y, handle), _as_rows(p, handle)) if save else _as_rows(y, handle)


def expert_linear_backward(grad_y, w, handle, p=None, stream=None):
    """Gradient of expert_linear w.r.t. its rows -> bf16 [rows, H]; with p, what
    the gated layer that made those rows saved, the gradient of p -> [rows,
    2H], which is that layer's grad_y."""
    rows, cap = _expert_rows(handle)
    g, w = _flat("grad_y", grad_y), _matrices(w)
    if w.dim() != 3:
        raise ValueError("w must be [E, N, H]")
    H = w.shape[2]
    grad_a = torch.empty((g.shape[0], 2 * H if p is not None else H), dtype=torch.bfloat16, device=grad_y.device)
    ep_expert_linear_backward(g, w, rows, cap, grad_a, _flat("p", p) if p is not None else None, stream)
    return _as_rows(grad_a, handle)


def expert_linear_backward_weights(grad_y, a, handle, dtype=torch.bfloat16, bias=False, stream=None):
    """Gradient of expert_linear w.r.t. its weights -> [E, N, H] of ``dtype``
    (bfloat16 or float32; [1, N, H] for ``handle`` None); with bias -> (grad_w,
    grad_bias [E, N]).  (ep_expert_linear_backward_weights adds to gradients
    that are there.)"""
    rows, cap = _expert_rows(handle)
    g, a2 = _flat("grad_y", grad_y), _flat("a", a)
    E = handle.num_experts if handle is not None else 1
    grad_w = torch.empty((E, g.shape[1], a2.shape[1]), dtype=dtype, device=grad_y.device)
    grad_bias = torch.empty((E, g.shape[1]), dtype=dtype, device=grad_y.device) if bias else None
    ep_expert_linear_backward_weights(g, a2, rows, cap, grad_w, grad_bias, False, stream)
    return (grad_w, grad_bias) if bias else grad_w
