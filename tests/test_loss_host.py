"""The objectives over logits on the CPU: the header compiles as C99 and agrees with the
binding's structures, bad arguments are refused before any launch, and the fp64 statements
that the GPU tests compare with have the gradient that differences give."""
import ctypes
import os
import re
import subprocess

import pytest

torch = pytest.importorskip("torch")

import loss_reference as R
import loss_scaled_adamw_gb300 as tl
from loss_scaled_adamw_gb300 import _build, losses

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
STRUCTS = (tl.tl_logits, tl.tl_loss_result, tl.tl_loss_out, tl.tl_policy_args, tl.tl_preference_args,
           tl.tl_distill_args)


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return losses._load()


def test_declared_functions_are_exported(lib):
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "tl_loss.h")).read(), flags=re.S)
    names = set(re.findall(r"\b(tl_[a-z_0-9]+)\s*\(", src))
    assert names == set(tl.LOSS_EXPORTED)
    for n in names:
        getattr(lib, n)


def test_c99_sees_the_binding_layout(tmp_path, lib):
    body = ['#include <stddef.h>', '#include <stdio.h>', '#include "tl_loss.h"', "typedef void (*any_fn)(void);",
            "int main(void) {"]
    for cls in STRUCTS:
        n = cls.__name__
        body.append(f'    printf("{n} %zu\\n", sizeof({n}));')
        body += [f'    printf("{n}.{f} %zu\\n", offsetof({n}, {f}));' for f, _ in cls._fields_]
    body.append("    any_fn fns[] = {" + ", ".join(f"(any_fn)&{n}" for n in tl.LOSS_EXPORTED) + "};")
    body += ['    printf("functions %zu\\n", sizeof(fns) / sizeof(fns[0]));', "    return 0;", "}"]
    src = tmp_path / "layout.c"
    src.write_text("\n".join(body))
    exe, where = str(tmp_path / "layout"), os.path.dirname(_build.LIB)
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Wextra", "-Werror", "-pedantic", "-I" + os.path.join(ROOT, "include"),
                    "-o", exe, str(src), "-L" + where, "-l:libtl_gb300.so", "-Wl,-rpath," + where],
                   check=True, capture_output=True, text=True)
    out = subprocess.run([exe], check=True, capture_output=True, text=True).stdout
    got = {k: int(v) for k, v in (line.rsplit(" ", 1) for line in out.strip().splitlines())}
    for cls in STRUCTS:
        assert got[cls.__name__] == ctypes.sizeof(cls)
        for f, _ in cls._fields_:
            assert got[f"{cls.__name__}.{f}"] == getattr(cls, f).offset, f
    assert got["functions"] == len(tl.LOSS_EXPORTED)


def test_null_contexts_and_bad_sizes_are_refused(lib):
    h = ctypes.c_void_p()
    assert lib.tl_loss_create(None, 1, 1, None) == tl.TL_EINVAL
    for rows, pairs in ((-1, 0), (1 << 31, 0), (1, -1), (1, (1 << 28) + 1)):
        assert lib.tl_loss_create(ctypes.byref(h), rows, pairs, None) == tl.TL_EINVAL and not h.value
    assert lib.tl_loss_destroy(None) == tl.TL_OK
    assert lib.tl_token_logprob(None, None, None, None, None) == tl.TL_EINVAL
    assert lib.tl_policy_loss(None, None, None, None, None) == tl.TL_EINVAL
    assert lib.tl_preference_loss(None, None, None, None, None) == tl.TL_EINVAL
    assert lib.tl_distill_loss(None, None, None, None, None) == tl.TL_EINVAL
    assert lib.tl_loss_launch_count(None) == 0 and lib.tl_loss_last_error(None) == b""


# ------------------------------------------------------------------ the fp64 statements

def _inputs(T, V, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, V, generator=g, dtype=torch.float64) * 1.5
    y = torch.randint(0, V, (T,), generator=g)
    y[T // 2] = -100
    return g, x, y


def checked_logits(loss, x, dx):
    """Central differences of `loss` at every element: step 1e-5, so the truncation error is
    about 1e-10 times a third derivative of order one and the rounding error 1e-16 / 1e-5."""
    num = torch.zeros_like(x)
    for t in range(x.shape[0]):
        for j in range(x.shape[1]):
            up, down = x.clone(), x.clone()
            up[t, j] += 1e-5
            down[t, j] -= 1e-5
            num[t, j] = (loss(up) - loss(down)) / 2e-5
    assert (num - dx).abs().max() < 1e-8


@pytest.mark.parametrize("tau", [1.0, 0.7, 2.0])
def test_policy_statement_has_the_gradient_of_its_loss(tau):
    g, x, y = _inputs(6, 5, 1)
    lp = R.logprob(x, y, tau)
    old = lp - torch.tensor([0.1, -0.1, 0.5, 0.0, -0.5, 0.5]).double()
    adv = torch.tensor([1.0, -2.0, 1.5, 3.0, -1.0, -0.5]).double()
    ref = lp + torch.randn(6, generator=g).double() * 0.3
    f = lambda v: float(R.policy(v, y, old, adv, 5, ref, kl_weight=0.3, tau=tau)["result"][0].double())  # noqa: E731
    loss = lambda v: R.policy(v, y, old, adv, 5, ref, kl_weight=0.3, tau=tau)["loss"].sum() / 5  # noqa: E731
    assert abs(f(x) - float(loss(x))) < 1e-6
    checked_logits(loss, x, R.policy(x, y, old, adv, 5, ref, kl_weight=0.3, tau=tau)["dx"])


@pytest.mark.parametrize("smooth", [0.0, 0.2])
def test_preference_statement_has_the_gradient_of_its_loss(smooth):
    g, x, y = _inputs(9, 4, 2)
    ref = torch.randn(9, generator=g).double()
    seq = [1, 3, 5, 5, 8]                       # rows 0 and 8 outside, an empty sequence
    loss = lambda v: R.preference(v, y, seq, 2, ref, 0.4, smooth, 1.3)["loss"].sum() / 2  # noqa: E731
    checked_logits(loss, x, R.preference(x, y, seq, 2, ref, 0.4, smooth, 1.3)["dx"])


@pytest.mark.parametrize("ce", [0.0, 0.5])
@pytest.mark.parametrize("tau", [1.0, 2.0])
def test_distill_statement_has_the_gradient_of_its_loss(tau, ce):
    g, x, y = _inputs(5, 6, 3)
    teacher = torch.randn(5, 3, generator=g).double()
    ids = torch.tensor([[0, 2, 5], [1, 1, 3], [4, 0, 1], [2, -1, 3], [-1, -1, -1]])
    loss = lambda v: R.distill(v, teacher, ids, 4, y, 0.7, ce, tau)["loss"].sum() / 4  # noqa: E731
    checked_logits(loss, x, R.distill(x, teacher, ids, 4, y, 0.7, ce, tau)["dx"])
