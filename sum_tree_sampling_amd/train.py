"""Thin Python binding of the C ABI in include/per_train.h: the operators a
learner that replays sequences runs next to the sum tree.

Functions carry the C names; sizes, types and strides come from the tensors.
Tensors must lie on the current device.  Outputs that are not given are
allocated on the stream the call runs on; with an explicit `stream` the usual
rule of torch holds for tensors used on another stream than their own: the
caller orders the streams and keeps the tensors alive (Tensor.record_stream).
Forward and backward passes are explicit calls; nothing is recorded for
autograd.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools

import torch

from .per import PerError, load

PER_F32, PER_BF16, PER_F16 = 0, 1, 2
PER_E4M3, PER_I8 = 0, 1
PER_SCAN_CHUNK = 64

_TYPE = {torch.float32: PER_F32, torch.bfloat16: PER_BF16, torch.float16: PER_F16}
_FORMAT = {torch.float8_e4m3fn: PER_E4M3, torch.int8: PER_I8}

_i64, _i32, _f64, _vp, _sz = (ctypes.c_int64, ctypes.c_int32, ctypes.c_double, ctypes.c_void_p,
                              ctypes.c_size_t)
_VIEW = [_vp, _i64, _i64]
_ROWS = [_i64, _i64, _i32, _i32, _vp, _i64, _vp, _i64]
_TOPK = [_i64, _i64, _i64, _i32, _vp, _i64, _vp, _vp, _i32, _vp, _f64]
_SIG = {
    "per_rows_write": _ROWS + [_i64, _i64, _vp, _i32, _i64, _vp],
    "per_rows_write_at": _ROWS + [_i64, _vp, _vp, _vp, _i32, _i64, _vp],
    "per_rows_read": _ROWS + [_i64, _vp, _i64, _vp, _i32, _i64, _vp],
    "per_scan_workspace_bytes": [_i64, _i64, _i64, ctypes.POINTER(_sz)],
    "per_scan_forward": [_i64, _i64, _i64, _i32] + 2 * _VIEW + [_vp, _vp, _vp] + _VIEW
    + [_vp, _vp, _vp, _sz, _vp],
    "per_scan_backward": [_i64, _i64, _i64, _i32] + 2 * _VIEW + [_vp, _vp, _vp] + _VIEW + [_vp]
    + 2 * _VIEW + [_vp, _vp, _sz, _vp],
    "per_scan_step": [_i64, _i64, _i32, _vp, _i64, _vp, _i64, _vp, _vp, _vp, _vp, _i64, _vp],
    "per_distill_workspace_bytes": [_i64, _i64, _i32, ctypes.POINTER(_sz)],
    "per_distill": _TOPK + [_vp, _vp, _vp, _i64, _vp, _sz, _vp],
    "per_distill_forward": _TOPK + [_vp, _vp, _vp, _sz, _vp],
    "per_distill_backward": _TOPK + [_vp, _vp, _vp, _i64, _vp],
}
_fn: dict = {}
_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _get(name):
    f = _fn.get(name)
    if f is None:
        f = getattr(load(), name)
        f.restype, f.argtypes = ctypes.c_int, _SIG[name]
        _fn[name] = f
    return f


def _fail(rc):
    raise PerError(rc, load().per_last_error().decode())


# ------------------------------------------------------------------ arguments
#
# The smallest calls take about as long on the host as on the device, so the
# checks below ask a tensor for as little as they can; what is wrong is found
# out only once something is.

def _need(ok, what):
    if not ok:
        raise ValueError(what)


def _current():
    """The current device, as tensors' get_device() gives it (which is -1 on the host)."""
    return _device() if torch.cuda.is_initialized() else -2


def _stream(stream, dev):
    if stream is None:
        return _raw_stream(dev) if _raw_stream else torch.cuda.current_stream(dev).cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _on(stream):
    """Allocations inside belong to the call's stream."""
    if stream is None:
        return contextlib.nullcontext()
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream))
    return torch.cuda.stream(stream)


def _empty(stream, shape, dtype, dev):
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    with _on(stream):
        return torch.empty(shape, dtype=dtype, device=dev)


def _refuse(t, name, dtype, shape, dev):
    _need(isinstance(t, torch.Tensor), "%s must be a tensor" % name)
    _need(t.get_device() == dev, "%s must be a tensor on the current device" % name)
    _need(t.dtype is dtype, "%s has type %s, expected %s" % (name, t.dtype, dtype))
    _need(tuple(t.shape) == tuple(shape),
          "%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
    _need(False, "%s must be contiguous" % name)


def _dense(t, name, dtype, shape, dev):
    """Pointer of a dense tensor of this type and shape (NULL for None)."""
    if t is None:
        return None
    if (t.dtype is not dtype or t.shape != shape or t.get_device() != dev
            or not t.is_contiguous()):
        _refuse(t, name, dtype, shape, dev)
    return t.data_ptr()


def _flags(t, name, shape, dev):
    return None if t is None else _dense(t, name, torch.uint8 if t.dtype is torch.uint8 else torch.bool,
                                         shape, dev)


def _row_stride(t, name):
    """Stride between the rows of a matrix with unit column stride."""
    s0, s1 = t.stride()
    n, d = t.shape
    if s1 != 1 and d > 1:
        raise ValueError("%s must have unit stride in its last dimension" % name)
    return s0 if n > 1 else max(d, s0)


def _matrix(t, name, dtype, shape, dev):
    """(pointer, row stride) of a matrix."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != dev:
        _refuse(t, name, dtype, shape, dev)
    return t.data_ptr(), _row_stride(t, name)


def _view(t, name, dtype, shape, dev):
    """(pointer, stride between sequences, between steps) of a [B x T x D] view."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != dev:
        _refuse(t, name, dtype, shape, dev)
    sb, st, sd = t.stride()
    if sd != 1 and shape[2] > 1:
        raise ValueError("%s must have unit stride in its last dimension" % name)
    return t.data_ptr(), sb, st


# ------------------------------------------------------------ 8-bit row store

def rows_alloc(capacity, dim, dtype=torch.float8_e4m3fn, group=128, device="cuda"):
    """A zeroed store: (codes [capacity x dim] of float8_e4m3fn or int8, scales
    [capacity x groups] f32), a row's scales behind its codes in one record."""
    _need(dtype in _FORMAT, "codes are float8_e4m3fn or int8")
    _need(group in (0, 32, 64, 128), "group is 0 (the row), 32, 64 or 128")
    ng = 1 if group == 0 else -(-dim // group)
    at = -(-dim // 4) * 4
    pitch = -(-(at + 4 * ng) // 16) * 16
    raw = torch.zeros(capacity, pitch, dtype=torch.uint8, device=device)
    return raw[:, :dim].view(dtype), raw.view(torch.float32)[:, at // 4:at // 4 + ng]


def _store(codes, scales, group, dev):
    fmt = _FORMAT.get(codes.dtype)
    if fmt is None or codes.dim() != 2:
        raise ValueError("codes must be [capacity x dim], float8_e4m3fn or int8")
    if group not in (0, 32, 64, 128):
        raise ValueError("group is 0 (the row), 32, 64 or 128")
    cap, dim = shape = codes.shape
    return (cap, dim, fmt, group, *_matrix(codes, "codes", codes.dtype, shape, dev),
            *_matrix(scales, "scales", torch.float32, (cap, -(-dim // group) if group else 1), dev))


def _source(src, dim, dev):
    t = _TYPE.get(src.dtype)
    if t is None or src.dim() != 2:
        raise ValueError("src must be [count x %d] of float32, bfloat16 or float16" % dim)
    p, st = _matrix(src, "src", src.dtype, (src.shape[0], dim), dev)
    return p, t, st


def per_rows_write(codes, scales, src, first=0, group=128, stream=None):
    """Quantise the rows of src into the ring's slots first, first + 1, ..."""
    dev = _current()
    st = _store(codes, scales, group, dev)
    rc = _get("per_rows_write")(*st, src.shape[0], first, *_source(src, st[1], dev),
                                _stream(stream, dev))
    if rc:
        _fail(rc)


def per_rows_write_at(codes, scales, src, slots, claims, group=128, stream=None):
    """Quantise row j of src into slot slots[j]; of a repeated slot the last
    position wins.  claims: [capacity] int32 zeros, zero again afterwards."""
    dev = _current()
    st = _store(codes, scales, group, dev)
    s = _source(src, st[1], dev)
    n = src.shape[0]
    rc = _get("per_rows_write_at")(*st, n, _dense(slots, "slots", torch.int64, (n,), dev),
                                   _dense(claims, "claims", torch.int32, (st[0],), dev), *s,
                                   _stream(stream, dev))
    if rc:
        _fail(rc)


def per_rows_read(codes, scales, idx, window=1, group=128, out=None, dtype=torch.float32,
                  stream=None):
    """[B x window x dim]: the rows of slots idx[b], idx[b] + 1, ... of the ring."""
    dev = _current()
    st = _store(codes, scales, group, dev)
    B, dim = idx.shape[0], st[1]
    _need(window >= 1, "window is at least 1")
    if out is None:
        out = _empty(stream, (B, window, dim), dtype, dev)
    t = _TYPE.get(out.dtype)
    _need(t is not None, "out has type %s" % out.dtype)
    rc = _get("per_rows_read")(*st, B, _dense(idx, "idx", torch.int64, (B,), dev), window,
                               _dense(out, "out", out.dtype, (B, window, dim), dev), t, dim,
                               _stream(stream, dev))
    if rc:
        _fail(rc)
    return out


# ----------------------------------------------------- gated linear recurrence

@functools.lru_cache(maxsize=1024)
def per_scan_workspace_bytes(B, T, D) -> int:
    out = _sz(0)
    rc = _get("per_scan_workspace_bytes")(B, T, D, ctypes.byref(out))
    if rc:
        _fail(rc)
    return out.value


def _seq(x, g, dev):
    t = _TYPE.get(x.dtype)
    if t is None or x.dim() != 3:
        raise ValueError("x must be [B x T x D] of float32, bfloat16 or float16")
    shape = x.shape
    return shape, t, _view(x, "x", x.dtype, shape, dev), _view(g, "g", x.dtype, shape, dev)


def per_scan_forward(x, g, reset=None, length=None, h0=None, y=None, h_last=None, carries=None,
                     stream=None):
    """h_t = f h_{t-1} + (1 - f) x_t with f = sigmoid(g_t) along dim 1 of x, g
    [B x T x D].  Returns (y [B x T x D], h_last [B x D] f32, carries: the f32
    states that per_scan_backward takes)."""
    dev = _current()
    shape, t, vx, vg = _seq(x, g, dev)
    B, T, D = shape
    f32 = torch.float32
    chunks = (B, -(-T // PER_SCAN_CHUNK), D)
    nbytes = per_scan_workspace_bytes(B, T, D)
    if y is None:
        y = _empty(stream, shape, x.dtype, dev)
    if h_last is None:
        h_last = _empty(stream, (B, D), f32, dev)
    if carries is None:
        carries = _empty(stream, chunks, f32, dev)
    ws = _empty(stream, nbytes, torch.uint8, dev) if nbytes else None
    rc = _get("per_scan_forward")(
        B, T, D, t, *vx, *vg, _flags(reset, "reset", (B, T), dev),
        _dense(length, "length", torch.int64, (B,), dev), _dense(h0, "h0", f32, (B, D), dev),
        *_view(y, "y", x.dtype, shape, dev), _dense(h_last, "h_last", f32, (B, D), dev),
        _dense(carries, "carries", f32, chunks, dev), ws.data_ptr() if nbytes else None, nbytes,
        _stream(stream, dev))
    if rc:
        _fail(rc)
    return y, h_last, carries


def per_scan_backward(x, g, carries, dy, reset=None, length=None, dh_last=None, dx=None, dg=None,
                      dh0=None, stream=None):
    """Gradients (dx, dg, dh0) of per_scan_forward from dy and dh_last."""
    dev = _current()
    shape, t, vx, vg = _seq(x, g, dev)
    B, T, D = shape
    f32 = torch.float32
    nbytes = per_scan_workspace_bytes(B, T, D)
    if dx is None:
        dx = _empty(stream, shape, x.dtype, dev)
    if dg is None:
        dg = _empty(stream, shape, x.dtype, dev)
    if dh0 is None:
        dh0 = _empty(stream, (B, D), f32, dev)
    ws = _empty(stream, nbytes, torch.uint8, dev) if nbytes else None
    rc = _get("per_scan_backward")(
        B, T, D, t, *vx, *vg, _flags(reset, "reset", (B, T), dev),
        _dense(length, "length", torch.int64, (B,), dev),
        _dense(carries, "carries", f32, (B, -(-T // PER_SCAN_CHUNK), D), dev),
        *_view(dy, "dy", x.dtype, shape, dev), _dense(dh_last, "dh_last", f32, (B, D), dev),
        *_view(dx, "dx", x.dtype, shape, dev), *_view(dg, "dg", x.dtype, shape, dev),
        _dense(dh0, "dh0", f32, (B, D), dev), ws.data_ptr() if nbytes else None, nbytes,
        _stream(stream, dev))
    if rc:
        _fail(rc)
    return dx, dg, dh0


def per_scan_step(x, g, h, reset=None, h_out=None, y=None, stream=None):
    """One step of B sequences: x, g [B x D], h [B x D] f32 (updated in place
    without h_out).  Returns (y, h_out)."""
    dev = _current()
    t = _TYPE.get(x.dtype)
    if t is None or x.dim() != 2:
        raise ValueError("x must be [B x D] of float32, bfloat16 or float16")
    dt, shape = x.dtype, x.shape
    mx, mg = _matrix(x, "x", dt, shape, dev), _matrix(g, "g", dt, shape, dev)
    if h_out is None:
        h_out = h
    if y is None:
        y = _empty(stream, shape, dt, dev)
    rc = _get("per_scan_step")(
        *shape, t, *mx, *mg,
        _flags(reset, "reset", shape[:1], dev), _dense(h, "h", torch.float32, shape, dev),
        _dense(h_out, "h_out", torch.float32, shape, dev), *_matrix(y, "y", dt, shape, dev),
        _stream(stream, dev))
    if rc:
        _fail(rc)
    return y, h_out


# ----------------------------------------------------------------- distillation

@functools.lru_cache(maxsize=1024)
def per_distill_workspace_bytes(N, V, type) -> int:  # noqa: A002
    out = _sz(0)
    rc = _get("per_distill_workspace_bytes")(N, V, type, ctypes.byref(out))
    if rc:
        _fail(rc)
    return out.value


def _top(logits, tidx, tlogit, tlse, temperature, dev):
    t = _TYPE.get(logits.dtype)
    if t is None or logits.dim() != 2 or tidx.dim() != 2:
        raise ValueError("logits must be [N x V] of float32, bfloat16 or float16, tidx [N x K]")
    N, V = shape = logits.shape
    top = (N, tidx.shape[1])
    tt = _TYPE.get(tlogit.dtype)
    _need(tt is not None, "tlogit has type %s" % tlogit.dtype)
    return (N, V, top[1], t, *_matrix(logits, "logits", logits.dtype, shape, dev),
            _dense(tidx, "tidx", torch.int32, top, dev), _dense(tlogit, "tlogit", tlogit.dtype, top, dev),
            tt, _dense(tlse, "tlse", torch.float32, (N,), dev), temperature)


def per_distill(logits, tidx, tlogit, tlse=None, temperature=1.0, weight=None, loss=None, grad=None,
                stream=None):
    """Per-row distillation loss [N] (not weighted) and its gradient by the
    logits [N x V] (weighted), against the teacher's logits tlogit [N x K] at
    tokens tidx [N x K] int32.  grad may be logits."""
    dev = _current()
    a = _top(logits, tidx, tlogit, tlse, temperature, dev)
    N, f32 = a[0], torch.float32
    nbytes = per_distill_workspace_bytes(N, a[1], a[3])
    if grad is None:
        grad = _empty(stream, logits.shape, logits.dtype, dev)
    if loss is None:
        loss = _empty(stream, (N,), f32, dev)
    ws = _empty(stream, nbytes, torch.uint8, dev) if nbytes else None
    rc = _get("per_distill")(
        *a, _dense(weight, "weight", f32, (N,), dev), _dense(loss, "loss", f32, (N,), dev),
        *_matrix(grad, "grad", logits.dtype, logits.shape, dev), ws.data_ptr() if nbytes else None,
        nbytes, _stream(stream, dev))
    if rc:
        _fail(rc)
    return loss, grad


def per_distill_forward(logits, tidx, tlogit, tlse=None, temperature=1.0, loss=None, saved=None,
                        stream=None):
    """Per-row loss [N], and the row statistics per_distill_backward takes."""
    dev = _current()
    a = _top(logits, tidx, tlogit, tlse, temperature, dev)
    N, f32 = a[0], torch.float32
    nbytes = per_distill_workspace_bytes(N, a[1], a[3])
    if loss is None:
        loss = _empty(stream, (N,), f32, dev)
    if saved is None:
        saved = _empty(stream, (N, 4), f32, dev)
    ws = _empty(stream, nbytes, torch.uint8, dev) if nbytes else None
    rc = _get("per_distill_forward")(
        *a, _dense(loss, "loss", f32, (N,), dev), _dense(saved, "saved", f32, (N, 4), dev),
        ws.data_ptr() if nbytes else None, nbytes, _stream(stream, dev))
    if rc:
        _fail(rc)
    return loss, saved


def per_distill_backward(logits, tidx, tlogit, saved, gloss, tlse=None, temperature=1.0, grad=None,
                         stream=None):
    """Gradient by the logits from the gradient by each row's loss."""
    dev = _current()
    a = _top(logits, tidx, tlogit, tlse, temperature, dev)
    N, f32 = a[0], torch.float32
    if grad is None:
        grad = _empty(stream, logits.shape, logits.dtype, dev)
    rc = _get("per_distill_backward")(
        *a, _dense(saved, "saved", f32, (N, 4), dev), _dense(gloss, "gloss", f32, (N,), dev),
        *_matrix(grad, "grad", logits.dtype, logits.shape, dev), _stream(stream, dev))
    if rc:
        _fail(rc)
    return grad
