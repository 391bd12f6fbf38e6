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

import ctypes

import torch

from .per import _check, _stream, load

PER_F32, PER_BF16, PER_F16 = 0, 1, 2
PER_E4M3, PER_I8 = 0, 1
PER_SCAN_CHUNK = 128

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


def _get(name):
    f = _fn.get(name)
    if f is None:
        f = getattr(load(), name)
        f.restype, f.argtypes = ctypes.c_int, _SIG[name]
        _fn[name] = f
    return f


# ------------------------------------------------------------------ arguments

def _need(ok, what):
    if not ok:
        raise ValueError(what)


def _on_device(t, name):
    _need(t.is_cuda and t.device.index == torch.cuda.current_device(),
          "%s must be a tensor on the current device" % name)


def _dense(t, name, dtype, *shape):
    """Pointer of a dense tensor of this type and shape (NULL for None)."""
    if t is None:
        return None
    _on_device(t, name)
    _need(t.dtype in dtype if isinstance(dtype, tuple) else t.dtype == dtype,
          "%s has type %s" % (name, t.dtype))
    _need(tuple(t.shape) == shape, "%s has shape %s, expected %s" % (name, tuple(t.shape), shape))
    _need(t.is_contiguous(), "%s must be contiguous" % name)
    return t.data_ptr()


def _row_stride(t, name):
    """Stride between the rows of a matrix with unit column stride."""
    n, d = t.shape
    _need(d <= 1 or t.stride(1) == 1, "%s must have unit stride in its last dimension" % name)
    return t.stride(0) if n > 1 else max(d, t.stride(0))


def _view(t, name, dtype, shape):
    """(pointer, stride between sequences, between steps) of a [B x T x D] view."""
    _on_device(t, name)
    _need(t.dtype == dtype, "%s has type %s, expected %s" % (name, t.dtype, dtype))
    _need(t.shape == shape, "%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
    s = t.stride()
    _need(shape[2] <= 1 or s[2] == 1, "%s must have unit stride in its last dimension" % name)
    return t.data_ptr(), s[0], s[1]


def _flags(t, name, *shape):
    return _dense(t, name, (torch.bool, torch.uint8), *shape)


class _On:
    """Allocations inside belong to the call's stream."""

    def __init__(self, stream):
        self.cm = None
        if stream is not None:
            s = stream
            if not isinstance(s, torch.cuda.Stream):
                s = torch.cuda.ExternalStream(int(s))
            self.cm = torch.cuda.stream(s)

    def __enter__(self):
        if self.cm is not None:
            self.cm.__enter__()

    def __exit__(self, *a):
        if self.cm is not None:
            self.cm.__exit__(*a)


def _scratch(nbytes, device):
    return torch.empty(nbytes, dtype=torch.uint8, device=device) if nbytes else None


def _ptr(t):
    return None if t is None else t.data_ptr()


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


def _store(codes, scales, group):
    _on_device(codes, "codes")
    _on_device(scales, "scales")
    fmt = _FORMAT.get(codes.dtype)
    _need(fmt is not None and codes.dim() == 2, "codes must be [capacity x dim], float8_e4m3fn or int8")
    _need(group in (0, 32, 64, 128), "group is 0 (the row), 32, 64 or 128")
    cap, dim = codes.shape
    ng = 1 if group == 0 else -(-dim // group)
    _need(scales.dtype == torch.float32 and tuple(scales.shape) == (cap, ng),
          "scales must be [capacity x %d] float32" % ng)
    return (cap, dim, fmt, group, codes.data_ptr(), _row_stride(codes, "codes"), scales.data_ptr(),
            _row_stride(scales, "scales"))


def _source(src, dim):
    _on_device(src, "src")
    t = _TYPE.get(src.dtype)
    _need(t is not None and src.dim() == 2 and src.shape[1] == dim,
          "src must be [count x %d] of float32, bfloat16 or float16" % dim)
    return src.data_ptr(), t, _row_stride(src, "src")


def per_rows_write(codes, scales, src, first=0, group=128, stream=None):
    """Quantise the rows of src into the ring's slots first, first + 1, ..."""
    st = _store(codes, scales, group)
    s = _source(src, st[1])
    _check(_get("per_rows_write")(*st, src.shape[0], int(first), *s, _stream(stream)))


def per_rows_write_at(codes, scales, src, slots, claims, group=128, stream=None):
    """Quantise row j of src into slot slots[j]; of a repeated slot the last
    position wins.  claims: [capacity] int32 zeros, zero again afterwards."""
    st = _store(codes, scales, group)
    s = _source(src, st[1])
    n = src.shape[0]
    _check(_get("per_rows_write_at")(*st, n, _dense(slots, "slots", torch.int64, n),
                                     _dense(claims, "claims", torch.int32, st[0]), *s,
                                     _stream(stream)))


def per_rows_read(codes, scales, idx, window=1, group=128, out=None, dtype=torch.float32,
                  stream=None):
    """[B x window x dim]: the rows of slots idx[b], idx[b] + 1, ... of the ring."""
    st = _store(codes, scales, group)
    _need(idx.dim() == 1, "idx must be [B]")
    B, window, dim = idx.shape[0], int(window), st[1]
    _need(window >= 1, "window is at least 1")
    p = _dense(idx, "idx", torch.int64, B)
    if out is None:
        with _On(stream):
            out = torch.empty(B, window, dim, dtype=dtype, device=codes.device)
    o, t = _dense(out, "out", (torch.float32, torch.bfloat16, torch.float16), B, window, dim), \
        _TYPE[out.dtype]
    _check(_get("per_rows_read")(*st, B, p, window, o, t, dim, _stream(stream)))
    return out


# ----------------------------------------------------- gated linear recurrence

def per_scan_workspace_bytes(B, T, D) -> int:
    out = _sz(0)
    _check(_get("per_scan_workspace_bytes")(int(B), int(T), int(D), ctypes.byref(out)))
    return out.value


def _seq(x, g):
    _need(x.dim() == 3, "x must be [B x T x D]")
    t = _TYPE.get(x.dtype)
    _need(t is not None, "x has type %s" % x.dtype)
    shape = x.shape
    return shape, t, _view(x, "x", x.dtype, shape), _view(g, "g", x.dtype, shape)


def per_scan_forward(x, g, reset=None, length=None, h0=None, y=None, h_last=None, carries=None,
                     stream=None):
    """h_t = f h_{t-1} + (1 - f) x_t with f = sigmoid(g_t) along dim 1 of x, g
    [B x T x D].  Returns (y [B x T x D], h_last [B x D] f32, carries: the f32
    states that per_scan_backward takes)."""
    shape, t, vx, vg = _seq(x, g)
    B, T, D = shape
    dev = x.device
    r, n = _flags(reset, "reset", B, T), _dense(length, "length", torch.int64, B)
    p0 = _dense(h0, "h0", torch.float32, B, D)
    nbytes = per_scan_workspace_bytes(B, T, D) if T > PER_SCAN_CHUNK else 0
    nch = -(-T // PER_SCAN_CHUNK)
    with _On(stream):
        if y is None:
            y = torch.empty(B, T, D, dtype=x.dtype, device=dev)
        if h_last is None:
            h_last = torch.empty(B, D, dtype=torch.float32, device=dev)
        if carries is None:
            carries = torch.empty(B, nch, D, dtype=torch.float32, device=dev)
        ws = _scratch(nbytes, dev)
    _check(_get("per_scan_forward")(
        B, T, D, t, *vx, *vg, r, n, p0, *_view(y, "y", x.dtype, shape),
        _dense(h_last, "h_last", torch.float32, B, D),
        _dense(carries, "carries", torch.float32, B, nch, D), _ptr(ws), nbytes, _stream(stream)))
    return y, h_last, carries


def per_scan_backward(x, g, carries, dy, reset=None, length=None, dh_last=None, dx=None, dg=None,
                      dh0=None, stream=None):
    """Gradients (dx, dg, dh0) of per_scan_forward from dy and dh_last."""
    shape, t, vx, vg = _seq(x, g)
    B, T, D = shape
    dev = x.device
    r, n = _flags(reset, "reset", B, T), _dense(length, "length", torch.int64, B)
    nbytes = per_scan_workspace_bytes(B, T, D) if T > PER_SCAN_CHUNK else 0
    c = _dense(carries, "carries", torch.float32, B, -(-T // PER_SCAN_CHUNK), D)
    vdy = _view(dy, "dy", x.dtype, shape)
    pl = _dense(dh_last, "dh_last", torch.float32, B, D)
    with _On(stream):
        if dx is None:
            dx = torch.empty(B, T, D, dtype=x.dtype, device=dev)
        if dg is None:
            dg = torch.empty(B, T, D, dtype=x.dtype, device=dev)
        if dh0 is None:
            dh0 = torch.empty(B, D, dtype=torch.float32, device=dev)
        ws = _scratch(nbytes, dev)
    _check(_get("per_scan_backward")(
        B, T, D, t, *vx, *vg, r, n, c, *vdy, pl, *_view(dx, "dx", x.dtype, shape),
        *_view(dg, "dg", x.dtype, shape), _dense(dh0, "dh0", torch.float32, B, D), _ptr(ws), nbytes,
        _stream(stream)))
    return dx, dg, dh0


def per_scan_step(x, g, h, reset=None, h_out=None, y=None, stream=None):
    """One step of B sequences: x, g [B x D], h [B x D] f32 (updated in place
    without h_out).  Returns (y, h_out)."""
    _need(x.dim() == 2 and x.dtype in _TYPE, "x must be [B x D] of float32, bfloat16 or float16")
    B, D = x.shape
    _on_device(x, "x")
    _on_device(g, "g")
    _need(g.shape == x.shape and g.dtype == x.dtype, "g must have the shape and type of x")
    if h_out is None:
        h_out = h
    if y is None:
        with _On(stream):
            y = torch.empty(B, D, dtype=x.dtype, device=x.device)
    _on_device(y, "y")
    _need(y.shape == x.shape and y.dtype == x.dtype, "y must have the shape and type of x")
    _check(_get("per_scan_step")(
        B, D, _TYPE[x.dtype], x.data_ptr(), _row_stride(x, "x"), g.data_ptr(), _row_stride(g, "g"),
        _flags(reset, "reset", B), _dense(h, "h", torch.float32, B, D),
        _dense(h_out, "h_out", torch.float32, B, D), y.data_ptr(), _row_stride(y, "y"),
        _stream(stream)))
    return y, h_out


# ----------------------------------------------------------------- distillation

def per_distill_workspace_bytes(N, V, type) -> int:  # noqa: A002
    out = _sz(0)
    _check(_get("per_distill_workspace_bytes")(int(N), int(V), int(type), ctypes.byref(out)))
    return out.value


def _top(logits, tidx, tlogit, tlse, temperature):
    _on_device(logits, "logits")
    _need(logits.dim() == 2 and logits.dtype in _TYPE,
          "logits must be [N x V] of float32, bfloat16 or float16")
    N, V = logits.shape
    _need(tidx.dim() == 2 and tidx.shape[0] == N, "tidx must be [N x K]")
    K = tidx.shape[1]
    return (N, V, K, _TYPE[logits.dtype], logits.data_ptr(), _row_stride(logits, "logits"),
            _dense(tidx, "tidx", torch.int32, N, K),
            _dense(tlogit, "tlogit", (torch.float32, torch.bfloat16, torch.float16), N, K),
            _TYPE[tlogit.dtype], _dense(tlse, "tlse", torch.float32, N), float(temperature))


def _grad(grad, logits, stream):
    if grad is None:
        with _On(stream):
            grad = torch.empty(logits.shape, dtype=logits.dtype, device=logits.device)
    _on_device(grad, "grad")
    _need(grad.shape == logits.shape and grad.dtype == logits.dtype,
          "grad must have the shape and type of logits")
    return grad, _row_stride(grad, "grad")


def per_distill(logits, tidx, tlogit, tlse=None, temperature=1.0, weight=None, loss=None, grad=None,
                stream=None):
    """Per-row distillation loss [N] (not weighted) and its gradient by the
    logits [N x V] (weighted), against the teacher's logits tlogit [N x K] at
    tokens tidx [N x K] int32.  grad may be logits."""
    a = _top(logits, tidx, tlogit, tlse, temperature)
    N = a[0]
    w = _dense(weight, "weight", torch.float32, N)
    grad, gs = _grad(grad, logits, stream)
    nbytes = per_distill_workspace_bytes(N, a[1], a[3])
    with _On(stream):
        if loss is None:
            loss = torch.empty(N, dtype=torch.float32, device=logits.device)
        ws = _scratch(nbytes, logits.device)
    _check(_get("per_distill")(*a, w, _dense(loss, "loss", torch.float32, N), grad.data_ptr(), gs,
                               _ptr(ws), nbytes, _stream(stream)))
    return loss, grad


def per_distill_forward(logits, tidx, tlogit, tlse=None, temperature=1.0, loss=None, saved=None,
                        stream=None):
    """Per-row loss [N], and the row statistics per_distill_backward takes."""
    a = _top(logits, tidx, tlogit, tlse, temperature)
    N = a[0]
    nbytes = per_distill_workspace_bytes(N, a[1], a[3])
    with _On(stream):
        if loss is None:
            loss = torch.empty(N, dtype=torch.float32, device=logits.device)
        if saved is None:
            saved = torch.empty(N, 4, dtype=torch.float32, device=logits.device)
        ws = _scratch(nbytes, logits.device)
    _check(_get("per_distill_forward")(*a, _dense(loss, "loss", torch.float32, N),
                                       _dense(saved, "saved", torch.float32, N, 4), _ptr(ws),
                                       nbytes, _stream(stream)))
    return loss, saved


def per_distill_backward(logits, tidx, tlogit, saved, gloss, tlse=None, temperature=1.0, grad=None,
                         stream=None):
    """Gradient by the logits from the gradient by each row's loss."""
    a = _top(logits, tidx, tlogit, tlse, temperature)
    N = a[0]
    grad, gs = _grad(grad, logits, stream)
    _check(_get("per_distill_backward")(*a, _dense(saved, "saved", torch.float32, N, 4),
                                        _dense(gloss, "gloss", torch.float32, N), grad.data_ptr(),
                                        gs, _stream(stream)))
    return grad
