"""The training objectives over vocabulary logits: Python binding of include/tl_loss.h.

Each call takes the logits of a micro-batch and writes its loss and, where asked for,
the gradient of the logits, multiplied by a scale that the device reads (the loss scale
S of a ``tl_create`` context, or the seed of ``tl_loss_seed``)::

    lctx = tl_loss_create(max_rows=4096, max_pairs=16)
    tl_policy_loss(lctx, logits, targets, old_logp, advantages, n_i, result,
                   seed=tl_scale_ptr(ctx), dlogits=dlogits)

The caller owns every tensor, outputs included; the binding checks and marshals them.
Logits and gradients are 2-D CUDA tensors [rows, vocab] whose rows are contiguous (any
row stride); per-row tensors are contiguous float32, targets and offsets int64.
``result`` is a float32 CUDA tensor of 4: loss, first and second term, count (see
``tl_loss_result``).  Tensors must stay alive, and be ordered with the call's stream,
until it has run.
"""
from __future__ import annotations

import ctypes
import sys

import torch

from . import TL_OK, TLError, _dropped, _release_dropped, load_library
from . import _stream as _any_stream

LOSS_EXPORTED = ("tl_loss_create", "tl_loss_destroy", "tl_token_logprob", "tl_policy_loss", "tl_preference_loss",
                 "tl_distill_loss", "tl_token_stats", "tl_token_grad", "tl_loss_launch_count", "tl_loss_last_error")

_vp, _i64, _i32, _f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float


class tl_logits(ctypes.Structure):
    _fields_ = [("data", _vp), ("rows", _i64), ("vocab", _i64), ("ld", _i64), ("dtype", _i32), ("temperature", _f32)]


class tl_loss_result(ctypes.Structure):
    _fields_ = [("loss", _f32), ("first", _f32), ("second", _f32), ("count", _f32)]


class tl_loss_out(ctypes.Structure):
    _fields_ = [("n", _i64), ("seed", _vp), ("dlogits", _vp), ("ld_dlogits", _i64), ("logp", _vp), ("loss", _vp),
                ("result", _vp)]


class tl_policy_args(ctypes.Structure):
    _fields_ = [("target", _vp), ("old_logp", _vp), ("ref_logp", _vp), ("advantage", _vp), ("clip_low", _f32),
                ("clip_high", _f32), ("kl_weight", _f32)]


class tl_preference_args(ctypes.Structure):
    _fields_ = [("target", _vp), ("seq", _vp), ("pairs", _i64), ("ref_logp", _vp), ("beta", _f32),
                ("label_smoothing", _f32), ("reward", _vp)]


class tl_distill_args(ctypes.Structure):
    _fields_ = [("target", _vp), ("teacher", _vp), ("teacher_id", _vp), ("ld_teacher", _i64), ("k", _i32),
                ("teacher_dtype", _i32), ("id_bytes", _i32), ("kd_weight", _f32), ("ce_weight", _f32)]


class tl_token_saved(ctypes.Structure):
    _fields_ = [("max", _f32), ("log_sum", _f32), ("entropy", _f32)]


class tl_token_stats_args(ctypes.Structure):
    _fields_ = [("target", _vp), ("logp", _vp), ("entropy", _vp), ("saved", _vp), ("top_id", _vp), ("top_logp", _vp),
                ("ld_top", _i64), ("k", _i32), ("id_bytes", _i32)]


class tl_token_grad_args(ctypes.Structure):
    _fields_ = [("target", _vp), ("saved", _vp), ("grad_logp", _vp), ("grad_entropy", _vp), ("seed", _vp),
                ("dlogits", _vp), ("ld_dlogits", _i64)]


_lib = _bind = None
_raw_stream = torch._C._cuda_getCurrentRawStream   # current_stream() without its Stream object (3 us a call)


def _stream(lctx, stream):
    """The raw stream of a call, as an integer: the current one of the context's device for None."""
    return _raw_stream(lctx.device) if stream is None else _any_stream(stream).value


def _load():
    """The library and the module that passes tensors to it (_loss_bind, csrc/tl_loss_bind.cpp)."""
    global _lib, _bind
    if _lib is None:
        lib = load_library()
        P = ctypes.POINTER
        for name, res, args in (
                ("tl_loss_create", ctypes.c_int, [P(_vp), _i64, _i64, _vp]),
                ("tl_loss_destroy", ctypes.c_int, [_vp]),
                ("tl_token_logprob", ctypes.c_int, [_vp, P(tl_logits), _vp, _vp, _vp]),
                ("tl_policy_loss", ctypes.c_int, [_vp, P(tl_logits), P(tl_policy_args), P(tl_loss_out), _vp]),
                ("tl_preference_loss", ctypes.c_int, [_vp, P(tl_logits), P(tl_preference_args), P(tl_loss_out), _vp]),
                ("tl_distill_loss", ctypes.c_int, [_vp, P(tl_logits), P(tl_distill_args), P(tl_loss_out), _vp]),
                ("tl_token_stats", ctypes.c_int, [_vp, P(tl_logits), P(tl_token_stats_args), _vp]),
                ("tl_token_grad", ctypes.c_int, [_vp, P(tl_logits), P(tl_token_grad_args), _vp]),
                ("tl_loss_launch_count", _i64, [_vp]),
                ("tl_loss_last_error", ctypes.c_char_p, [_vp])):
            fn = getattr(lib, name)
            fn.restype, fn.argtypes = res, args
        try:
            from . import _loss_bind as _bind
        except ImportError as e:
            raise ImportError("loss_scaled_adamw_gb300/_loss_bind.so is missing: build it with "
                              "loss_scaled_adamw_gb300._build.build(); there is no fallback") from e
        _lib = lib
    return _lib


class LossContext:
    """Owns one tl_loss_ctx (its scratch lives on the device that was current at creation).  Dropped without
    tl_loss_destroy, its scratch is released by the next create or destroy of a context."""

    def __init__(self, handle, device: int):
        self.handle = handle
        self.device = device

    @property
    def _address(self):
        return self.handle.value if self.handle else None

    def __del__(self):
        if getattr(self, "handle", None) and _lib is not None and not sys.is_finalizing():
            _dropped.append((_lib.tl_loss_destroy, self.handle))
            self.handle = None


def _check(lctx, fn: str, rc: int):
    if rc != TL_OK:
        detail = _lib.tl_loss_last_error(lctx.handle).decode() if lctx.handle else "the context has been destroyed"
        raise TLError(fn, rc, detail or _lib.tl_status_string(rc).decode())


def tl_loss_create(max_rows: int, max_pairs: int = 0, stream=None) -> LossContext:
    """A context for calls of at most max_rows rows and max_pairs preference pairs."""
    lib = _load()
    _release_dropped()
    h = _vp()
    rc = lib.tl_loss_create(ctypes.byref(h), int(max_rows), int(max_pairs), _any_stream(stream))
    if rc != TL_OK:
        raise TLError("tl_loss_create", rc, lib.tl_status_string(rc).decode())
    return LossContext(h, torch.cuda.current_device())


def tl_loss_destroy(lctx: LossContext) -> None:
    if lctx.handle:
        rc = _load().tl_loss_destroy(lctx.handle)
        lctx.handle = None
        _release_dropped()
        if rc != TL_OK:
            raise TLError("tl_loss_destroy", rc)


def tl_loss_launch_count(lctx: LossContext) -> int:
    return int(_load().tl_loss_launch_count(lctx.handle))


def tl_token_logprob(lctx: LossContext, logits, targets, logp, temperature: float = 1.0, stream=None) -> None:
    """logp[t] = log softmax(logits[t] / temperature)[targets[t]]; 0 where targets[t] < 0."""
    rc = _bind.token_logprob(lctx._address, lctx.device, logits, temperature, targets, logp, _stream(lctx, stream))
    if rc != TL_OK:
        _check(lctx, "tl_token_logprob", rc)


def tl_policy_loss(lctx: LossContext, logits, targets, old_logp, advantages, n: int, result, ref_logp=None,
                   clip_low: float = 0.2, clip_high: float = 0.2, kl_weight: float = 0.0, temperature: float = 1.0,
                   seed=None, dlogits=None, logp=None, row_loss=None, stream=None) -> None:
    """Clipped policy objective with a KL penalty, mean over n valid targets; its gradient
    into dlogits (which may be the logits themselves).  seed: a device address (tl_scale_ptr),
    a float32 CUDA tensor of one element, or None (a gradient of the plain mean)."""
    rc = _bind.policy_loss(lctx._address, lctx.device, logits, temperature, n, seed, dlogits, logp, row_loss, result,
                           _stream(lctx, stream), targets, old_logp, ref_logp, advantages, clip_low, clip_high,
                           kl_weight)
    if rc != TL_OK:
        _check(lctx, "tl_policy_loss", rc)


def tl_preference_loss(lctx: LossContext, logits, targets, seq, n: int, result, ref_logp=None, beta: float = 0.1,
                       label_smoothing: float = 0.0, temperature: float = 1.0, seed=None, dlogits=None, logp=None,
                       pair_loss=None, reward=None, stream=None) -> None:
    """Paired preference objective, mean over n pairs.  seq: int64 CUDA tensor of
    2 * pairs + 1 row offsets (chosen, rejected, chosen, ...)."""
    rc = _bind.preference_loss(lctx._address, lctx.device, logits, temperature, n, seed, dlogits, logp, pair_loss,
                               result, _stream(lctx, stream), targets, seq, ref_logp, beta, label_smoothing, reward)
    if rc != TL_OK:
        _check(lctx, "tl_preference_loss", rc)


def tl_distill_loss(lctx: LossContext, logits, teacher_logits, teacher_ids, n: int, result, targets=None,
                    kd_weight: float = 1.0, ce_weight: float = 0.0, temperature: float = 1.0, seed=None, dlogits=None,
                    row_loss=None, stream=None) -> None:
    """Distillation from a teacher's top-k logits ([rows, k], ids int32 or int64), mean over
    n valid rows.  teacher_logits = teacher_ids = None is the cross-entropy alone."""
    rc = _bind.distill_loss(lctx._address, lctx.device, logits, temperature, n, seed, dlogits, None, row_loss, result,
                            _stream(lctx, stream), targets, teacher_logits, teacher_ids, kd_weight, ce_weight)
    if rc != TL_OK:
        _check(lctx, "tl_distill_loss", rc)


def tl_token_stats(lctx: LossContext, logits, targets=None, logp=None, entropy=None, top_ids=None, top_logp=None,
                   saved=None, temperature: float = 1.0, stream=None) -> None:
    """Log-probabilities of the targets, entropies, and the k likeliest alternatives of each
    row ([rows, k]: ids int32 or int64, and their log-probabilities, the likeliest first and
    the lower id first among equal logits).  saved ([rows, 3]: largest logit, log of the sum
    of exponentials against it, entropy) is what tl_token_grad takes.  The alternatives are
    what tl_distill_loss takes as a teacher's logits and ids."""
    rc = _bind.token_stats(lctx._address, lctx.device, logits, temperature, targets, logp, entropy, saved, top_ids,
                           top_logp, _stream(lctx, stream))
    if rc != TL_OK:
        _check(lctx, "tl_token_stats", rc)


def tl_token_grad(lctx: LossContext, logits, saved, dlogits, targets=None, grad_logp=None, grad_entropy=None,
                  temperature: float = 1.0, seed=None, stream=None) -> None:
    """dlogits (which may be the logits themselves) = the gradient of seed times
    sum_t grad_logp[t] * logp[t] + grad_entropy[t] * entropy[t], with saved of tl_token_stats
    for the same logits and temperature.  seed as for tl_policy_loss."""
    rc = _bind.token_grad(lctx._address, lctx.device, logits, temperature, saved, dlogits, targets, grad_logp,
                          grad_entropy, seed, _stream(lctx, stream))
    if rc != TL_OK:
        _check(lctx, "tl_token_grad", rc)
