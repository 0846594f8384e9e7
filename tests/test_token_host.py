"""Row statistics, their gradient and dropout on the CPU: the headers compile as C99 and agree with the
binding's structures, bad arguments are refused before any launch, the fp64 statements have the gradient that
differences give, and the random numbers are the published generator's."""
import ctypes
import os
import re
import subprocess

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import loss_scaled_adamw_gb300 as tl
import token_reference as R
from loss_scaled_adamw_gb300 import _build, losses

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
STRUCTS = (tl.tl_token_saved, tl.tl_token_stats_args, tl.tl_token_grad_args, tl.tl_dropout_args)


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return losses._load()


def test_dropout_is_declared_and_exported(lib):
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "tl_dropout.h")).read(), flags=re.S)
    assert set(re.findall(r"\b(tl_[a-z_0-9]+)\s*\(", src)) == set(tl.DROPOUT_EXPORTED)
    for n in tl.DROPOUT_EXPORTED:
        getattr(lib, n)


def test_c99_sees_the_binding_layout(tmp_path):
    body = ['#include <stddef.h>', '#include <stdio.h>', '#include "tl_loss.h"', '#include "tl_dropout.h"', "int main(void) {"]
    for cls in STRUCTS:
        n = cls.__name__
        body.append(f'    printf("{n} %zu\\n", sizeof({n}));')
        body += [f'    printf("{n}.{f} %zu\\n", offsetof({n}, {f}));' for f, _ in cls._fields_]
    src, exe = tmp_path / "layout.c", str(tmp_path / "layout")
    src.write_text("\n".join(body + ["    return 0;", "}"]))
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Wextra", "-Werror", "-pedantic", "-I" + os.path.join(ROOT, "include"),
                    "-o", exe, str(src)], check=True, capture_output=True, text=True)
    out = subprocess.run([exe], check=True, capture_output=True, text=True).stdout
    got = {k: int(v) for k, v in (line.rsplit(" ", 1) for line in out.strip().splitlines())}
    for cls in STRUCTS:
        assert got[cls.__name__] == ctypes.sizeof(cls)
        for f, _ in cls._fields_:
            assert got[f"{cls.__name__}.{f}"] == getattr(cls, f).offset, f


def test_null_contexts_are_refused(lib):
    assert lib.tl_token_stats(None, None, None, None) == tl.TL_EINVAL
    assert lib.tl_token_grad(None, None, None, None) == tl.TL_EINVAL


BASE = 1 << 40   # fake device addresses: nothing is launched


def _dropout_args(**kw):
    a = dict(x=BASE, residual=None, y=BASE + (1 << 30), rows=4, cols=100, ldx=100, ldr=0, ldy=100, key=BASE - 4096, site=1,
             dtype=tl.TL_BF16, p=0.5, device=12345)
    a.update(kw)
    return tl.tl_dropout_args(**a)


def test_dropout_refuses_bad_arguments(lib):
    lib.tl_dropout.restype, lib.tl_dropout.argtypes = ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p]
    call = lambda **kw: lib.tl_dropout(ctypes.byref(_dropout_args(**kw)), None)  # noqa: E731
    # valid arguments get as far as the device: none here, or another one
    assert call() in (tl.TL_ECUDA, tl.TL_ESTATE)
    assert call(y=BASE) in (tl.TL_ECUDA, tl.TL_ESTATE)                                    # in place
    assert call(y=BASE + 200, ldx=200, ldy=200) in (tl.TL_ECUDA, tl.TL_ESTATE)            # columns beside x's
    assert lib.tl_dropout(None, None) == tl.TL_EINVAL
    bad = [dict(dtype=3), dict(dtype=-1), dict(p=-0.1), dict(p=1.5), dict(p=float("nan")), dict(rows=-1), dict(cols=-1),
           dict(rows=1 << 22, cols=1 << 22, ldx=1 << 22, ldy=1 << 22), dict(key=None), dict(key=BASE + 4), dict(x=None),
           dict(y=None), dict(x=BASE + 1), dict(ldx=99), dict(ldy=99), dict(ldx=1 << 40), dict(y=BASE + 2),
           dict(y=BASE, ldy=101), dict(residual=BASE + (1 << 20), ldr=99), dict(residual=BASE + (1 << 30) + 2, ldr=100),
           dict(key=BASE + (1 << 30) + 8), dict(y=BASE + 100, ldx=120, ldy=120)]
    for kw in bad:
        assert call(**kw) == tl.TL_EINVAL, kw


# ------------------------------------------------------------------ the fp64 statements

@pytest.mark.parametrize("tau", [1.0, 0.7, 2.0])
def test_gradient_formula_against_differences(tau):
    g = torch.Generator().manual_seed(3)
    T, V = 5, 11
    x = torch.randn(T, V, generator=g, dtype=torch.float64) * 2
    x[3, 4] = -R.INF
    y = torch.tensor([2, 0, -100, 7, 10])
    ga, gb = torch.randn(T, generator=g), torch.randn(T, generator=g)

    def value(x):
        s = R.stats(x, y, 0, tau)
        return float((ga.double() * s["logp"] + gb.double() * s["entropy"])[y >= 0].sum())

    d, h = R.grad(x, y, ga, gb, tau), 1e-6
    for t in range(T):
        for j in range(V):
            if x[t, j] == -R.INF:
                assert d[t, j] == 0
                continue
            up, down = x.clone(), x.clone()
            up[t, j] += h
            down[t, j] -= h
            assert abs((value(up) - value(down)) / (2 * h) - float(d[t, j])) < 1e-8


def test_statistics_statement():
    s = R.stats(torch.zeros(1, 8), torch.tensor([3]), 3)
    assert abs(float(s["entropy"]) - np.log(8)) < 1e-15 and s["ids"].tolist() == [[0, 1, 2]]
    x = torch.tensor([[1.0, -R.INF, 3.0, 3.0], [R.NAN, 0, 0, 0], [-R.INF] * 4, [R.INF, 0, 0, 0]])
    s = R.stats(x, torch.tensor([2, 1, 1, 9]), 4)
    assert s["ids"].tolist() == [[2, 3, 0, -1]] + [[-1] * 4] * 3
    assert s["top"][0, 3] == -R.INF and torch.isnan(s["top"][1:]).all() and torch.isnan(s["logp"][1:]).all()


def test_generator_known_answers():
    """The published known-answer vectors of Philox4x32-10."""
    assert R.philox([0] * 4, (0, 0)) == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    assert R.philox([0xFFFFFFFF] * 4, (0xFFFFFFFF, 0xFFFFFFFF)) == [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]
    assert R.philox([0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344], (0xA4093822, 0x299F31D0)) == \
        [0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1]


def test_numbers_of_a_stretch_are_the_generators():
    seed, ticket, site = -7, (5 << 32) + 9, 11
    w = R.philox([3, 5 << 8, 9, 11], (seed % 2 ** 32, seed % 2 ** 64 >> 32))
    want = [h for v in w for h in (v & 0xFFFF, v >> 16)]
    assert R.numbers(24, 8, seed, ticket, site).tolist() == want
    assert R.numbers(26, 3, seed, ticket, site).tolist() == want[2:5]
    n = R.numbers(0, 1 << 16, seed, ticket, site)
    assert abs(n.mean() / 65536 - 0.5) < 5 * 0.2887 / 256      # five standard deviations
