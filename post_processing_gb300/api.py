"""PyTorch-tensor front end of the C ABI (marshalling only).

Tensors supply device memory, pinned host memory and streams; every result
is computed by ``libws.so`` on the GPU.
"""
from __future__ import annotations

from typing import NamedTuple

import torch

from . import binding as B


# the current stream of a device as an integer: torch's own accessor where it has one, as it costs a thirtieth of
# making a Stream object
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda device: torch.cuda.current_stream(device).cuda_stream)


_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _elsewhere(device: int, name: str) -> ValueError:
    """A call runs on its main operand's device, which has to be the current one, as the library launches there."""
    return ValueError(f"{name} is on cuda:{device}, the current device is cuda:{_current_device()}")


def _other_stream(stream, device: int):
    """The stream of a call's `stream` argument (a Stream or a raw one), None where it is the device's current one."""
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream)) if int(stream) else torch.cuda.default_stream()
    if getattr(stream, "device_index", device) != device:
        raise ValueError(f"the stream belongs to cuda:{stream.device_index}, the call runs on cuda:{device}")
    return None if stream.cuda_stream == _current_stream(device) else stream


def _empty(shape, dtype, device) -> torch.Tensor:
    return torch.empty(shape, dtype=dtype, device=device)


def _results(other, make, *args):
    """make(*args): a call's results.  For a call on another stream they come from that stream's memory: a block of the current
    stream's may still be read by work queued there under its last owner.  They are held for both streams."""
    if other is None:
        return make(*args)
    with torch.cuda.stream(other):
        out = make(*args)
    current = torch.cuda.current_stream()
    for t in out if isinstance(out, tuple) else (out,):
        if t is not None:
            t.record_stream(current)
    return out


def _held(other, *tensors) -> int:
    """The raw handle of a stream other than the current one, for whose work the tensors' memory is held."""
    for t in tensors:
        if t is not None:
            t.record_stream(other)
    return other.cuda_stream


def preprocess(frames: torch.Tensor, desc: B.ws_preprocess_desc, batch: int | None = None,
               out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """ws_preprocess on a uint8 CUDA tensor holding `batch` frames."""
    if frames.dtype != torch.uint8 or not frames.is_cuda:
        raise TypeError("frames must be a uint8 CUDA tensor")
    if batch is None:
        batch = frames.shape[0]
    device = frames.get_device()
    if device != _current_device():
        raise _elsewhere(device, "frames")
    other = None if stream is None else _other_stream(stream, device)
    if out is None:
        dtype = {B.WS_DTYPE_F32: torch.float32, B.WS_DTYPE_F16: torch.float16,
                 B.WS_DTYPE_BF16: torch.bfloat16}[desc.dst_type]
        out = _results(other, _empty, (batch, 3, desc.dst_h, desc.dst_w), dtype, frames.device)
    B.check(B.ws_preprocess(desc, frames.data_ptr(), batch, out.data_ptr(),
                            _current_stream(device) if other is None else _held(other, frames, out)))
    return out


def _workspace(n: int, device, stream):
    """n bytes at a 256-byte boundary, and the raw stream of a call's `stream` argument, from whose memory they come."""
    index = torch.device(device).index
    if index not in (None, _current_device()):
        raise _elsewhere(index, "a workspace")
    index = _current_device()
    other = None if stream is None else _other_stream(stream, index)
    ws = _results(other, _empty, (n + 256,), torch.uint8, device)
    off = (-ws.data_ptr()) % 256
    return ws[off:off + n], _current_stream(index) if other is None else other.cuda_stream


def topk_workspace(rows: int, cols: int, k: int, device="cuda", stream=None) -> torch.Tensor | None:
    """A zeroed workspace for ws_topk of this shape (None when none is needed)."""
    st, n = B.ws_topk_workspace_bytes(rows, cols, k)
    B.check(st)
    if n == 0:
        return None
    ws, raw = _workspace(n, device, stream)
    B.check(B.ws_topk_workspace_init(ws.data_ptr(), n, raw))
    return ws


def topk(x: torch.Tensor, k: int, out_val: torch.Tensor | None = None, out_idx: torch.Tensor | None = None,
         workspace: torch.Tensor | None = None, stream=None):
    """ws_topk on a float32 CUDA tensor [rows, cols] (or [cols])."""
    if x.dtype != torch.float32 or not x.is_cuda or not x.is_contiguous():
        raise TypeError("x must be a contiguous float32 CUDA tensor")
    rows, cols = (1, x.shape[0]) if x.dim() == 1 else x.shape
    device = x.get_device()
    if device != _current_device():
        raise _elsewhere(device, "x")
    other = None if stream is None else _other_stream(stream, device)
    if out_val is None:
        out_val = _results(other, _empty, (rows, k), torch.float32, x.device)
    if out_idx is None:
        out_idx = _results(other, _empty, (rows, k), torch.int32, x.device)
    if workspace is None:
        workspace = topk_workspace(rows, cols, k, x.device, stream)
    wptr, wbytes = (workspace.data_ptr(), workspace.numel()) if workspace is not None else (None, 0)
    B.check(B.ws_topk(x.data_ptr(), rows, cols, k, out_val.data_ptr(), out_idx.data_ptr(), wptr, wbytes,
                      _current_stream(device) if other is None else _held(other, x, out_val, out_idx, workspace)))
    return out_val, out_idx


_DTYPES = {torch.float32: B.WS_DTYPE_F32, torch.float16: B.WS_DTYPE_F16, torch.bfloat16: B.WS_DTYPE_BF16}
_INDEX_TYPES = {torch.int32: B.WS_INDEX_I32, torch.int64: B.WS_INDEX_I64}


class Logprobs(NamedTuple):
    """What logprobs() gives, per row: the token's log probability (None without tokens), the entropy, the
    log-sum-exp, the sums that logprobs_backward() takes, and the k likeliest entries (None for k = 0)."""
    logprob: torch.Tensor | None
    entropy: torch.Tensor
    lse: torch.Tensor
    stats: torch.Tensor
    top_logprob: torch.Tensor | None
    top_idx: torch.Tensor | None


class Distill(NamedTuple):
    """What distill() gives: the weighted loss of each row, and the gradient of the logits (None without it)."""
    loss: torch.Tensor
    grad: torch.Tensor | None


def _matrix(x: torch.Tensor, name: str):
    """(rows, cols, row stride, type, device) of a CUDA tensor [rows, cols] whose rows are contiguous, or [cols]."""
    dtype, device = _DTYPES.get(x.dtype), x.get_device()
    if dtype is None or device < 0:
        raise TypeError(f"{name} must be a float32, float16 or bfloat16 CUDA tensor")
    shape = x.shape
    if len(shape) == 2:
        rows, cols = shape
        stride, step = x.stride()
        if rows == 1:
            stride = cols
    elif len(shape) == 1:
        rows, cols = 1, shape[0]
        stride, step = cols, x.stride(0)
    else:
        raise TypeError(f"{name} must be [rows, cols] or [cols]")
    if step != 1 and cols > 1:
        raise TypeError(f"{name}'s rows must be contiguous")
    return rows, cols, stride, dtype, device


def _operand(t: torch.Tensor | None, name: str, shape: tuple, dtypes, device: int):
    """The address of a contiguous tensor of this shape and one of these types on this device (None for None)."""
    if t is None:
        return None
    if t.get_device() == device and t.dtype in dtypes and t.shape == shape and t.is_contiguous():
        return t.data_ptr()
    if t.dtype not in dtypes or not t.is_cuda or not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous CUDA tensor of {' or '.join(str(d) for d in dtypes)}")
    if t.shape != shape:
        raise ValueError(f"{name} is {tuple(t.shape)}, {shape} expected")
    raise ValueError(f"{name} is on another device than the call's cuda:{device}")


_F32, _I32 = (torch.float32,), (torch.int32,)


def _new_logprobs(rows: int, k: int, with_tokens: bool, device) -> Logprobs:
    """Results in one allocation (each tensor contiguous)."""
    logprob, entropy, lse, stats, top = torch.empty(rows * (5 + k), dtype=torch.float32, device=device).split(
        (rows, rows, rows, 2 * rows, k * rows))
    return Logprobs(logprob if with_tokens else None, entropy, lse, stats.view(rows, 2), top.view(rows, k) if k else None,
                    torch.empty((rows, k), dtype=torch.int32, device=device) if k else None)


def _spent(logits: torch.Tensor) -> None:
    """Logits that were overwritten by their gradient: autograd is told, so that a graph that saved them says so when it
    is run backward, in place of using what is there now."""
    torch.autograd.graph.increment_version(logits)


def _new_distill(rows: int, logits: torch.Tensor, grad: bool) -> Distill:
    return Distill(_empty((rows,), torch.float32, logits.device),
                   _empty(logits.shape, logits.dtype, logits.device) if grad else None)


def logprobs(logits: torch.Tensor, tokens: torch.Tensor | None = None, k: int = 0, temperature: float = 1.0,
             out: Logprobs | None = None, stream=None) -> Logprobs:
    """ws_logprobs on a CUDA tensor [rows, cols] (or [cols]) of float32, float16 or bfloat16, whose rows may be
    padded.  tokens: int32 or int64 [rows], negative where a row has none.  out: an earlier result of the same
    call to write into.

    Results carry no autograd history, whether or not the logits require a gradient: a loss on them is
    differentiated by logprobs_backward(), whose gradient goes on by logits.backward(gradient)."""
    rows, cols, stride, dtype, device = _matrix(logits, "logits")
    if device != _current_device():
        raise _elsewhere(device, "logits")
    other = None if stream is None else _other_stream(stream, device)
    if out is None:
        out = _results(other, _new_logprobs, rows, k, tokens is not None, logits.device)
    per_row = (rows,)
    tok = _operand(tokens, "tokens", per_row, _INDEX_TYPES, device)
    desc = B.ws_logprobs_desc(rows, cols, stride, dtype, _INDEX_TYPES[tokens.dtype] if tokens is not None else 0, k,
                              temperature)
    status = B.ws_logprobs(desc, logits.data_ptr(), tok, _operand(out.logprob, "out.logprob", per_row, _F32, device),
                           _operand(out.entropy, "out.entropy", per_row, _F32, device),
                           _operand(out.lse, "out.lse", per_row, _F32, device),
                           _operand(out.stats, "out.stats", (rows, 2), _F32, device),
                           _operand(out.top_logprob, "out.top_logprob", (rows, k), _F32, device),
                           _operand(out.top_idx, "out.top_idx", (rows, k), _I32, device),
                           _current_stream(device) if other is None else _held(other, logits, tokens, *out))
    if status:
        B.check(status)
    return out


def logprobs_backward(logits: torch.Tensor, tokens: torch.Tensor | None, stats: torch.Tensor,
                      entropy: torch.Tensor | None, grad_logprob: torch.Tensor | None,
                      grad_entropy: torch.Tensor | None = None, temperature: float = 1.0,
                      out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """ws_logprobs_backward: the gradient of the logits from those of logprobs()' log probabilities and entropies
    (either may be None); stats and entropy as logprobs() gave them.  out: a tensor of the logits' shape and type
    whose rows may be padded, the logits themselves included (they are spent then, and autograd's version of them
    counts up); other rows that overlap the logits' are refused."""
    rows, cols, stride, dtype, device = _matrix(logits, "logits")
    if device != _current_device():
        raise _elsewhere(device, "logits")
    other = None if stream is None else _other_stream(stream, device)
    if out is None:
        out = _results(other, _empty, logits.shape, logits.dtype, logits.device)
    out_rows, out_cols, out_stride, out_dtype, where = _matrix(out, "out")
    if where != device:
        raise ValueError(f"out is on another device than the call's cuda:{device}")
    if (out_rows, out_cols, out_dtype) != (rows, cols, dtype):
        raise ValueError("out has another shape or type than the logits")
    per_row = (rows,)
    desc = B.ws_logprobs_desc(rows, cols, stride, dtype, _INDEX_TYPES.get(tokens.dtype, 0) if tokens is not None else 0,
                              0, temperature)
    at, to = logits.data_ptr(), out.data_ptr()
    status = B.ws_logprobs_backward(desc, at, _operand(tokens, "tokens", per_row, _INDEX_TYPES, device),
                                    _operand(stats, "stats", (rows, 2), _F32, device),
                                    _operand(entropy, "entropy", per_row, _F32, device),
                                    _operand(grad_logprob, "grad_logprob", per_row, _F32, device),
                                    _operand(grad_entropy, "grad_entropy", per_row, _F32, device), to, out_stride,
                                    _current_stream(device) if other is None else _held(
                                        other, logits, tokens, stats, entropy, grad_logprob, grad_entropy, out))
    if status:
        B.check(status)
    if to == at:
        _spent(out)
    return out


def distill(logits: torch.Tensor, teacher_idx: torch.Tensor, teacher_logprob: torch.Tensor,
            weight: torch.Tensor | None = None, temperature: float = 1.0, tail: bool = False, grad: bool = True,
            out: Distill | None = None, stream=None) -> Distill:
    """ws_distill on a student's logits [rows, cols] and a teacher's top entries [rows, k] (logprobs()' top_idx and
    top_logprob; int32 or int64 indices).  tail: the teacher's remaining mass is one more class, else its entries
    are renormalised.  weight: float32 [rows].  out: a Distill to write into (its grad may be the logits,
    as for logprobs_backward()).  The loss carries no autograd history; the gradient goes on by
    logits.backward(grad)."""
    rows, cols, stride, dtype, device = _matrix(logits, "logits")
    if teacher_idx.dim() != logits.dim():
        raise ValueError("teacher_idx must have as many dimensions as the logits")
    k = teacher_idx.shape[-1]
    if device != _current_device():
        raise _elsewhere(device, "logits")
    other = None if stream is None else _other_stream(stream, device)
    if out is None:
        out = _results(other, _new_distill, rows, logits, grad)
    gptr, gstride = None, cols
    if out.grad is not None:
        g_rows, g_cols, gstride, g_dtype, where = _matrix(out.grad, "out.grad")
        if where != device:
            raise ValueError(f"out.grad is on another device than the call's cuda:{device}")
        if (g_rows, g_cols, g_dtype) != (rows, cols, dtype):
            raise ValueError("out.grad has another shape or type than the logits")
        gptr = out.grad.data_ptr()
    entries = (rows, k) if logits.dim() == 2 else (k,)
    ids = _operand(teacher_idx, "teacher_idx", entries, _INDEX_TYPES, device)
    desc = B.ws_distill_desc(rows, cols, stride, gstride, dtype, _INDEX_TYPES[teacher_idx.dtype], k,
                             B.WS_DISTILL_TAIL if tail else B.WS_DISTILL_RENORM, temperature)
    at = logits.data_ptr()
    status = B.ws_distill(desc, at, ids,
                          _operand(teacher_logprob, "teacher_logprob", entries, _F32, device),
                          _operand(weight, "weight", (rows,), _F32, device),
                          _operand(out.loss, "out.loss", (rows,), _F32, device), gptr, _current_stream(device) if other is None else
                          _held(other, logits, teacher_idx, teacher_logprob, weight, *out))
    if status:
        B.check(status)
    if gptr == at:
        _spent(out.grad)
    return out


def detect_workspace(desc: B.ws_detect_desc, batch: int, device="cuda", stream=None) -> torch.Tensor:
    """A zeroed, 256-byte aligned workspace for ws_detect of this geometry and batch."""
    st, n = B.ws_detect_workspace_bytes(desc, batch)
    B.check(st)
    ws, raw = _workspace(n, device, stream)
    B.check(B.ws_detect_workspace_init(ws.data_ptr(), n, raw))
    return ws


def detect(head: torch.Tensor, desc: B.ws_detect_desc, workspace: torch.Tensor | None = None,
           out: torch.Tensor | None = None, out_count: torch.Tensor | None = None, stream=None):
    """ws_detect on a float32 CUDA head [batch, 4*reg_max + num_classes, A].

    Returns (detections, counts): detections is the raw int32 [batch, max_det,
    8] buffer of ws_detection records and counts the int32 [batch] kept per
    image; detection_fields() gives named views of it."""
    if head.dtype != torch.float32 or not head.is_cuda or not head.is_contiguous() or head.dim() != 3:
        raise TypeError("head must be a contiguous float32 CUDA tensor [batch, channels, anchors]")
    batch = head.shape[0]
    device = head.get_device()
    if device != _current_device():
        raise _elsewhere(device, "head")
    other = None if stream is None else _other_stream(stream, device)
    if workspace is None:
        workspace = detect_workspace(desc, batch, head.device, stream)
    if out is None:
        out = _results(other, _empty, (batch, desc.max_det, 8), torch.int32, head.device)
    if out_count is None:
        out_count = _results(other, _empty, (batch,), torch.int32, head.device)
    B.check(B.ws_detect(desc, head.data_ptr(), batch, out.data_ptr(), out_count.data_ptr(), workspace.data_ptr(),
                        workspace.numel(),
                        _current_stream(device) if other is None else _held(other, head, out, out_count, workspace)))
    return out, out_count


def detection_fields(detections: torch.Tensor) -> dict:
    """Named views of a [..., 8] int32 ws_detection buffer: boxes (x1, y1, x2,
    y2) and score as float32, class and anchor as int32."""
    f = detections.view(torch.float32)
    return {"boxes": f[..., 0:4], "score": f[..., 4], "cls": detections[..., 5], "anchor": detections[..., 6]}


class Pool:
    """ws_pool_*: N identical lanes with a producer / consumer hand-off;
    destroyed by close() or `with`.  Lanes are returned as raw handles."""

    def __init__(self, desc: B.ws_lane_desc, lanes: int):
        st, h = B.ws_pool_create(desc, lanes)
        B.check(st)
        self.handle = h
        self.size = lanes
        self._batch = desc.batch

    def lane(self, i: int) -> int:
        st, h = B.ws_pool_lane(self.handle, i)
        B.check(st)
        return h

    def buffers(self, lane: int) -> B.ws_lane_buffers:
        st, b = B.ws_lane_get_buffers(lane)
        B.check(st)
        return b

    def acquire(self, timeout_us: int = -1) -> int | None:
        """A free lane, or None if none became free in time (back-pressure)."""
        st, h = B.ws_pool_acquire(self.handle, timeout_us)
        if st == B.WS_ERR_TIMEOUT:
            return None
        B.check(st)
        return h

    def submit(self, lane: int, n: int | None = None):
        """Submit the lane's whole batch, or its first n frames."""
        B.check(B.ws_pool_submit(self.handle, lane, self._batch if n is None else n))

    def complete(self, timeout_us: int = -1):
        """(lane, timing) of the oldest submission, or (None, None) on timeout."""
        st, h, t = B.ws_pool_complete(self.handle, timeout_us)
        if st == B.WS_ERR_TIMEOUT:
            return None, None
        B.check(st)
        return h, t

    def recycle(self, lane: int):
        B.check(B.ws_pool_recycle(self.handle, lane))

    def close(self):
        if self.handle is not None:
            B.check(B.ws_pool_destroy(self.handle))
            self.handle = None

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()


class Lane:
    """One fixed-shape lane (ws_lane_*); destroyed by close() or `with`."""

    def __init__(self, desc: B.ws_lane_desc):
        st, h = B.ws_lane_create(desc)
        B.check(st)
        self.handle = h
        st, self.buffers = B.ws_lane_get_buffers(h)
        B.check(st)

    def acquire(self):
        B.check(B.ws_lane_acquire(self.handle))

    def submit(self, n: int | None = None):
        """Submit the whole batch, or the first n frames (ws_lane_submit_n)."""
        B.check(B.ws_lane_submit(self.handle) if n is None else B.ws_lane_submit_n(self.handle, n))

    def rebind(self, input: int | None = None, logits: int | None = None) -> bool:
        """Point the lane at new slots; True if a graph was re-instantiated."""
        st, re = B.ws_lane_rebind(self.handle, input, logits)
        B.check(st)
        st, self.buffers = B.ws_lane_get_buffers(self.handle)
        B.check(st)
        return bool(re)

    def wait(self, timeout_us: int = -1) -> B.ws_lane_timing:
        st, t = B.ws_lane_wait(self.handle, timeout_us)
        B.check(st)
        return t

    def release(self):
        B.check(B.ws_lane_release(self.handle))

    @property
    def state(self) -> int:
        return B.ws_lane_state(self.handle)

    def close(self):
        if self.handle is not None:
            B.check(B.ws_lane_destroy(self.handle))
            self.handle = None

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()
