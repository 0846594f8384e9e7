"""Dropout whose mask is never stored: Python binding of include/tl_dropout.h.

The mask is a function of a key on the device ([seed, ticket], int64), of the site (which
dropout of the model) and of an element's place in its tensor, so the backward pass, and a
micro-batch that is computed again, see it by naming the same key::

    key = torch.tensor([seed, 0], dtype=torch.int64, device="cuda")
    tl_dropout(branch, hidden, 0.1, key, site=3, residual=hidden)    # hidden += dropout(branch)
    ...
    tl_dropout(d_hidden, d_branch, 0.1, key, site=3)                 # the gradient of branch
    key[1] += 1                                                      # the next micro-batch's ticket

All of it can be captured in a CUDA graph: a replay reads the key anew.
"""
from __future__ import annotations

import ctypes

import torch

from . import TL_OK, TLError, losses

DROPOUT_EXPORTED = ("tl_dropout", "tl_dropout_last_error")

_vp, _i64, _i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32


class tl_dropout_args(ctypes.Structure):
    _fields_ = [("x", _vp), ("residual", _vp), ("y", _vp), ("rows", _i64), ("cols", _i64), ("ldx", _i64), ("ldr", _i64),
                ("ldy", _i64), ("key", _vp), ("site", ctypes.c_uint32), ("dtype", _i32), ("p", ctypes.c_float),
                ("device", _i32)]


def tl_dropout(x, y, p: float, key, site: int = 0, residual=None, stream=None) -> None:
    """y = residual + (kept ? x / (1 - p) : 0), p to the nearest multiple of 2^-16.

    x, y and residual: float32, bfloat16 or float16 CUDA tensors of one shape and dtype,
    contiguous, or 2-D with contiguous rows.  y may be x or the residual itself.  The
    gradient of x is the same call on the gradient of y, without a residual."""
    bind = losses._bind
    if bind is None:
        losses._load()
        bind = losses._bind
    device = x.get_device() if isinstance(x, torch.Tensor) else -1
    if device < 0:
        raise ValueError("x must be a CUDA tensor")
    handle = losses._raw_stream(device) if stream is None else losses._any_stream(stream).value
    rc = bind.dropout(x, y, residual, key, site, p, handle, device)
    if rc != TL_OK:
        last_error = losses._load().tl_dropout_last_error
        last_error.restype, last_error.argtypes = ctypes.c_char_p, []
        raise TLError("tl_dropout", rc, last_error().decode())
