"""Sizes beyond a grid of 2^31 CTAs are refused as an argument, with a text that names them.  The addresses are not of
any memory: such sizes are in no launch's reach."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

import loss_scaled_adamw_gb300 as tl
from loss_scaled_adamw_gb300 import losses

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lctx():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from loss_scaled_adamw_gb300 import _build
    _build.build()
    return tl.tl_loss_create(2 ** 31 - 1)


@pytest.mark.parametrize("vocab,dtype", [(1 << 14, tl.TL_BF16), (1 << 14, tl.TL_F32), (1 << 20, tl.TL_F16)])
def test_gradient_of_more_logits_than_a_grid_takes(lctx, vocab, dtype):
    lib, rows, x = losses._load(), 2 ** 31 - 1, 1 << 56
    logits = tl.tl_logits(x, rows, vocab, vocab, dtype, 1.0)
    args = tl.tl_token_grad_args(target=None, saved=1 << 40, grad_logp=None, grad_entropy=1 << 44, seed=None, dlogits=x,
                                 ld_dlogits=vocab)
    before = tl.tl_loss_launch_count(lctx)
    rc = lib.tl_token_grad(lctx.handle, ctypes.byref(logits), ctypes.byref(args), None)
    assert rc == tl.TL_EINVAL and b"rows * vocab" in lib.tl_loss_last_error(lctx.handle)
    assert tl.tl_loss_launch_count(lctx) == before
