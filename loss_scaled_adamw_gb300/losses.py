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
import struct

import torch

from . import TL_BF16, TL_F16, TL_F32, TL_OK, TLError, load_library
from . import _stream as _any_stream

LOSS_EXPORTED = ("tl_loss_create", "tl_loss_destroy", "tl_token_logprob", "tl_policy_loss", "tl_preference_loss",
                 "tl_distill_loss", "tl_loss_launch_count", "tl_loss_last_error")

_DTYPES = {torch.float32: TL_F32, torch.bfloat16: TL_BF16, torch.float16: TL_F16}
_ID_BYTES = {torch.int32: 4, torch.int64: 8}
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


_lib = None
_raw_stream = torch._C._cuda_getCurrentRawStream   # current_stream() without its Stream object (3 us a call)


def _stream(lctx, stream):
    return _raw_stream(lctx.device) if stream is None else _any_stream(stream)


def _load():
    global _lib
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
                ("tl_loss_launch_count", _i64, [_vp]),
                ("tl_loss_last_error", ctypes.c_char_p, [_vp])):
            fn = getattr(lib, name)
            fn.restype, fn.argtypes = res, args
        _lib = lib
    return _lib


class LossContext:
    """Owns one tl_loss_ctx (its scratch lives on the device that was current at creation)
    and the argument structures that its calls fill in (a context is used by one thread)."""

    def __init__(self, handle, device: int):
        self.handle = handle
        self.device = device
        self._x, self._out = tl_logits(), tl_loss_out()
        self._args = {c: c() for c in (tl_policy_args, tl_preference_args, tl_distill_args)}
        # one pack per call and structure: assigning the fields one by one costs more than
        # the launch
        self._refs = {c: ctypes.byref(v) for c, v in self._args.items()}
        self._x_ref, self._out_ref = ctypes.byref(self._x), ctypes.byref(self._out)

    def __del__(self):
        if getattr(self, "handle", None) and _lib is not None:
            _lib.tl_loss_destroy(self.handle)
            self.handle = None


# The structures' layouts for struct.pack_into (native sizes and alignment).
_PACK_LOGITS = struct.Struct("@Pqqqif")
_PACK_OUT = struct.Struct("@qPPqPPP")
_PACK = {tl_policy_args: struct.Struct("@PPPPfff"), tl_preference_args: struct.Struct("@PPqPffP"),
         tl_distill_args: struct.Struct("@PPPqiiiff")}


def _check(lctx, fn: str, rc: int):
    if rc != TL_OK:
        detail = _lib.tl_loss_last_error(lctx.handle).decode() if lctx.handle else "the context has been destroyed"
        raise TLError(fn, rc, detail or _lib.tl_status_string(rc).decode())


def tl_loss_create(max_rows: int, max_pairs: int = 0, stream=None) -> LossContext:
    """A context for calls of at most max_rows rows and max_pairs preference pairs."""
    lib = _load()
    h = _vp()
    rc = lib.tl_loss_create(ctypes.byref(h), int(max_rows), int(max_pairs), _any_stream(stream))
    if rc != TL_OK:
        raise TLError("tl_loss_create", rc, lib.tl_status_string(rc).decode())
    return LossContext(h, torch.cuda.current_device())


def tl_loss_destroy(lctx: LossContext) -> None:
    if lctx.handle:
        rc = _load().tl_loss_destroy(lctx.handle)
        lctx.handle = None
        if rc != TL_OK:
            raise TLError("tl_loss_destroy", rc)


def tl_loss_launch_count(lctx: LossContext) -> int:
    return int(_load().tl_loss_launch_count(lctx.handle))


_F32, _I64 = torch.float32, torch.int64


def _vec(lctx, t, dtype, n: int, name: str) -> int:
    """Address of a contiguous device vector of n elements, 0 for None."""
    if t is None:
        return 0
    if t.dtype is not dtype or t.numel() != n or not t.is_contiguous() or t.get_device() != lctx.device:
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of {n} elements on cuda:{lctx.device}")
    return t.data_ptr()


def _matrix(lctx, t, name: str):
    """(address, rows, columns, row stride) of a 2-D device tensor with contiguous rows."""
    if t.dim() != 2 or t.get_device() != lctx.device:
        raise ValueError(f"{name} must be a 2-D tensor on cuda:{lctx.device}")
    rows, cols = t.shape
    ld, step = t.stride()
    if step != 1 and cols > 1:
        raise ValueError(f"the rows of {name} must be contiguous")
    return t.data_ptr(), rows, cols, ld if rows > 1 or ld > cols else cols


def _logits(lctx, x, temperature) -> int:
    """Fills in the context's tl_logits; the number of rows."""
    addr, rows, vocab, ld = _matrix(lctx, x, "logits")
    dt = _DTYPES.get(x.dtype)
    if dt is None:
        raise ValueError("logits must be float32, bfloat16 or float16")
    _PACK_LOGITS.pack_into(lctx._x, 0, addr, rows, vocab, ld, dt, temperature)
    return rows


def _out(lctx, x, n, result, seed, dlogits, logp, rows, loss, losses) -> None:
    """Fills in the context's tl_loss_out.  seed: a device address (tl_scale_ptr), a float32
    CUDA tensor of one element, or None."""
    d = ldd = 0
    if dlogits is not None:
        d, _, _, ldd = _matrix(lctx, dlogits, "dlogits")
        if dlogits.dtype is not x.dtype or dlogits.shape != x.shape:
            raise ValueError("dlogits must have the shape and dtype of the logits")
    if not isinstance(seed, int):
        seed = _vec(lctx, seed, _F32, 1, "seed")
    _PACK_OUT.pack_into(lctx._out, 0, n, seed, d, ldd, _vec(lctx, logp, _F32, rows, "logp"),
                        _vec(lctx, loss, _F32, losses, "the loss output"), _vec(lctx, result, _F32, 4, "result"))


def _call(lctx, name: str, cls, stream, *fields) -> None:
    _PACK[cls].pack_into(lctx._args[cls], 0, *fields)
    rc = getattr(_load(), name)(lctx.handle, lctx._x_ref, lctx._refs[cls], lctx._out_ref, _stream(lctx, stream))
    if rc != TL_OK:
        _check(lctx, name, rc)


def tl_token_logprob(lctx: LossContext, logits, targets, logp, temperature: float = 1.0, stream=None) -> None:
    """logp[t] = log softmax(logits[t] / temperature)[targets[t]]; 0 where targets[t] < 0."""
    T = _logits(lctx, logits, temperature)
    rc = _load().tl_token_logprob(lctx.handle, lctx._x_ref, _vec(lctx, targets, _I64, T, "targets"),
                                  _vec(lctx, logp, _F32, T, "logp"), _stream(lctx, stream))
    if rc != TL_OK:
        _check(lctx, "tl_token_logprob", rc)


def tl_policy_loss(lctx: LossContext, logits, targets, old_logp, advantages, n: int, result, ref_logp=None,
                   clip_low: float = 0.2, clip_high: float = 0.2, kl_weight: float = 0.0, temperature: float = 1.0,
                   seed=None, dlogits=None, logp=None, row_loss=None, stream=None) -> None:
    """Clipped policy objective with a KL penalty, mean over n valid targets; its gradient
    into dlogits (which may be the logits themselves)."""
    T = _logits(lctx, logits, temperature)
    _out(lctx, logits, n, result, seed, dlogits, logp, T, row_loss, T)
    _call(lctx, "tl_policy_loss", tl_policy_args, stream, _vec(lctx, targets, _I64, T, "targets"),
          _vec(lctx, old_logp, _F32, T, "old_logp"), _vec(lctx, ref_logp, _F32, T, "ref_logp"),
          _vec(lctx, advantages, _F32, T, "advantages"), clip_low, clip_high, kl_weight)


def tl_preference_loss(lctx: LossContext, logits, targets, seq, n: int, result, ref_logp=None, beta: float = 0.1,
                       label_smoothing: float = 0.0, temperature: float = 1.0, seed=None, dlogits=None, logp=None,
                       pair_loss=None, reward=None, stream=None) -> None:
    """Paired preference objective, mean over n pairs.  seq: int64 CUDA tensor of
    2 * pairs + 1 row offsets (chosen, rejected, chosen, ...)."""
    T = _logits(lctx, logits, temperature)
    bounds = seq.numel()
    if bounds % 2 != 1:
        raise ValueError("seq must hold 2 * pairs + 1 offsets")
    pairs = bounds // 2
    _out(lctx, logits, n, result, seed, dlogits, logp, T, pair_loss, pairs)
    _call(lctx, "tl_preference_loss", tl_preference_args, stream, _vec(lctx, targets, _I64, T, "targets"),
          _vec(lctx, seq, _I64, bounds, "seq"), pairs, _vec(lctx, ref_logp, _F32, T, "ref_logp"), beta,
          label_smoothing, _vec(lctx, reward, _F32, 2 * pairs, "reward"))


def tl_distill_loss(lctx: LossContext, logits, teacher_logits, teacher_ids, n: int, result, targets=None,
                    kd_weight: float = 1.0, ce_weight: float = 0.0, temperature: float = 1.0, seed=None, dlogits=None,
                    row_loss=None, stream=None) -> None:
    """Distillation from a teacher's top-k logits ([rows, k], ids int32 or int64), mean over
    n valid rows.  teacher_logits = teacher_ids = None is the cross-entropy alone."""
    T = _logits(lctx, logits, temperature)
    t_addr = i_addr = ldt = k = tdt = id_bytes = 0
    if teacher_logits is not None:
        t_addr, t_rows, k, ldt = _matrix(lctx, teacher_logits, "teacher_logits")
        i_addr, i_rows, i_cols, ldi = _matrix(lctx, teacher_ids, "teacher_ids")
        tdt = _DTYPES.get(teacher_logits.dtype, -1)
        id_bytes = _ID_BYTES.get(teacher_ids.dtype, -1)
        if t_rows != T or i_rows != T or i_cols != k or ldt != ldi:
            raise ValueError("teacher_logits and teacher_ids must be [rows, k] with one row stride")
    _out(lctx, logits, n, result, seed, dlogits, None, T, row_loss, T)
    _call(lctx, "tl_distill_loss", tl_distill_args, stream, _vec(lctx, targets, _I64, T, "targets"), t_addr, i_addr,
          ldt, k, tdt, id_bytes, kd_weight, ce_weight)
