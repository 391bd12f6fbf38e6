"""Thin Python binding of the C ABI in include/per_train.h: the operators a
learner that replays sequences runs next to the sum tree.

Functions carry the C names; sizes, types and strides come from the tensors
(csrc/marshal.cpp checks them and raises ValueError, or PerError with the
library's own text).  Tensors must lie on the current device.  Outputs that are
not given are allocated on the stream the call runs on; with an explicit
`stream` the usual rule of torch holds for tensors used on another stream than
their own: the caller orders the streams and keeps the tensors alive
(Tensor.record_stream).  Forward and backward passes are explicit calls;
nothing is recorded for autograd.  Any argument that requires grad is refused
while autograd records (not under no_grad, nor inside an autograd.Function), and
any that carries a forward-mode tangent while those are taken.  Tensors that a
call writes count as changed in place (Tensor._version).
"""
from __future__ import annotations

import ctypes

import torch

from .per import PerError, load

PER_F32, PER_BF16, PER_F16 = 0, 1, 2
PER_E4M3, PER_I8 = 0, 1
PER_SCAN_CHUNK = 64

NAMES = ("per_rows_write", "per_rows_write_at", "per_rows_read", "per_scan_workspace_bytes",
         "per_scan_forward", "per_scan_backward", "per_scan_step", "per_distill_workspace_bytes",
         "per_distill", "per_distill_forward", "per_distill_backward")


def _bind():
    """Hand the library's entry points to the binding (at its first call)."""
    lib = load()
    _marshal.bind({n: ctypes.cast(getattr(lib, n), ctypes.c_void_p).value
                   for n in NAMES + ("per_last_error",)}, PerError)


def _missing(name):
    def f(*args, **kwargs):
        raise ImportError("_marshal.so is not built or failed to load; run "
                          "sum_tree_sampling_amd.build.build()") from _why
    f.__name__ = name
    return f


try:
    from . import _marshal
    _marshal.set_loader(_bind)
    globals().update({n: getattr(_marshal, n) for n in NAMES})
except ImportError as e:  # before the first build; the calls say so
    _why = e
    globals().update({n: _missing(n) for n in NAMES})


def rows_alloc(capacity, dim, dtype=torch.float8_e4m3fn, group=128, device="cuda"):
    """A zeroed store: (codes [capacity x dim] of float8_e4m3fn or int8, scales
    [capacity x groups] f32), a row's scales behind its codes in one record."""
    if dtype not in (torch.float8_e4m3fn, torch.int8):
        raise ValueError("codes are float8_e4m3fn or int8")
    if group not in (0, 32, 64, 128):
        raise ValueError("group is 0 (the row), 32, 64 or 128")
    ng = 1 if group == 0 else -(-dim // group)
    at = -(-dim // 4) * 4
    pitch = -(-(at + 4 * ng) // 16) * 16
    raw = torch.zeros(capacity, pitch, dtype=torch.uint8, device=device)
    return raw[:, :dim].view(dtype), raw.view(torch.float32)[:, at // 4:at // 4 + ng]
