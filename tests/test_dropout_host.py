"""Arguments of dropout on the CPU, where the checks that every call makes end before the device is asked."""
import ctypes
import os
import subprocess
import sys

import pytest

pytest.importorskip("torch")

import loss_scaled_adamw_gb300 as tl
import test_token_host as H
from loss_scaled_adamw_gb300 import _build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_one_row_has_no_stride():
    """In a child process: a stride times the element size that wraps to 0 has been divided by."""
    _build.build()
    code = """
import sys; sys.path[:0] = [%r, %r]
import ctypes, test_token_host as H, loss_scaled_adamw_gb300 as tl
from loss_scaled_adamw_gb300 import losses
lib = losses._load()
lib.tl_dropout.restype, lib.tl_dropout.argtypes = ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p]
call = lambda **kw: lib.tl_dropout(ctypes.byref(H._dropout_args(rows=1, dtype=tl.TL_F32, **kw)), None)
ok, far = (tl.TL_ECUDA, tl.TL_ESTATE), 1 << 62
assert call(y=H.BASE + 8, ldx=far, ldy=far) == tl.TL_EINVAL           # overlaps x, 8 bytes on
assert call(y=H.BASE + 396, ldx=far, ldy=far) == tl.TL_EINVAL
assert call(y=H.BASE + 400, ldx=far, ldy=far) in ok                   # behind x
assert call(y=H.BASE, ldx=far, ldy=far) in ok                         # in place
assert call(y=H.BASE, ldx=120, ldy=100) in ok                         # in place, whatever the strides
assert call(x=H.BASE + 4096, y=H.BASE, residual=H.BASE, ldr=1000, ldy=100) in ok
assert call(x=H.BASE + 4096, y=H.BASE, residual=H.BASE + 4, ldr=100, ldy=100) == tl.TL_EINVAL
assert call(y=H.BASE, ldx=99, ldy=100) == tl.TL_EINVAL
""" % (ROOT, os.path.join(ROOT, "tests"))
    subprocess.run([sys.executable, "-c", code], check=True, timeout=300)


lib = H.lib


def test_more_elements_than_a_grid_takes_are_refused(lib):
    """As an argument, not as a failed launch."""
    lib.tl_dropout.restype, lib.tl_dropout.argtypes = ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p]
    for cols, ok in ((1 << 20, True), ((1 << 20) + 1, False), (1 << 21, False), (1 << 23, False)):
        args = H._dropout_args(rows=1 << 20, cols=cols, ldx=cols + 1, ldy=cols + 1, y=H.BASE + (1 << 46))
        rc = lib.tl_dropout(ctypes.byref(args), None)
        assert rc in (tl.TL_ECUDA, tl.TL_ESTATE) if ok else rc == tl.TL_EINVAL, cols


def test_errors_name_the_argument(lib):
    lib.tl_dropout.restype, lib.tl_dropout.argtypes = ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p]
    lib.tl_dropout_last_error.restype, lib.tl_dropout_last_error.argtypes = ctypes.c_char_p, []
    far = H.BASE + (1 << 30)
    for word, kw in ((b"dtype", dict(dtype=7)), (b"p must", dict(p=2.0)), (b"rows", dict(rows=-1)), (b"key must", dict(key=None)),
                     (b"x must", dict(ldx=99)), (b"y must", dict(y=None)), (b"residual must", dict(residual=far + 1, ldr=100)),
                     (b"y overlaps x", dict(y=H.BASE + 2)), (b"y overlaps residual", dict(residual=far + 2, ldr=100)),
                     (b"y overlaps key", dict(key=far + 8))):
        assert lib.tl_dropout(ctypes.byref(H._dropout_args(**kw)), None) == tl.TL_EINVAL
        assert word in lib.tl_dropout_last_error(), (word, lib.tl_dropout_last_error())
    assert lib.tl_dropout(None, None) == tl.TL_EINVAL and b"args" in lib.tl_dropout_last_error()
