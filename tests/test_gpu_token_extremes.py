"""Row statistics and their gradient on the GPU where products and differences of logits leave fp32: temperatures next to
the limits, and the largest and the lowest value of a type in one row.  Results are those of the fp64 statement, rounded
to fp32 (a log-probability beyond it is -inf); tolerances are those of test_gpu_token.py."""
import pytest

torch = pytest.importorskip("torch")

import test_gpu_token as G
import token_reference as R

pytestmark = pytest.mark.gpu

lctx = G.lctx
INF = float("inf")


def in_fp32(want):
    return {n: v if n == "ids" else v.float().double() for n, v in want.items()}


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("V,times", [(40, 1), (1003, 300), (9000, 1), (20001, 1), (33000, 60)])
@pytest.mark.parametrize("tau", [2.0 ** -33, 1.3e-20, 2.0 ** -126])
def test_temperatures_next_to_zero(lctx, V, times, dtype, tau):
    """The largest entries, three equal ones, share the row; all others are far below, or excluded."""
    x = torch.full((4, V), -1.0, dtype=G.DT[dtype])
    x[0, :: 2] = -INF
    x[1, ::3] = torch.finfo(x.dtype).min
    x[2, 4:20] = torch.finfo(x.dtype).min / 4
    x[3, V // 2:] = -2.0 ** -10
    for row in range(4):
        x[row, [1, 7, V - 1]] = 0.0
    y = torch.tensor([1, 7, 2, V - 1])
    for k in (0, 3):
        _, got = G.run(lctx, x.repeat(times, 1), y.repeat(times), k, tau)
        want = in_fp32(R.stats(x, y, k, torch.tensor(tau).double()))
        G.compare(got, {n: v.repeat(times, *[1] * (v.dim() - 1)) for n, v in want.items()})


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("V,times", [(40, 1), (1003, 300), (9000, 1), (20001, 1), (20001, 60), (33000, 60)])
@pytest.mark.parametrize("tau", [2.0 ** 100, 2.0 ** 126])
def test_excluded_entries_at_temperatures_next_to_infinity(lctx, V, times, dtype, tau):
    """Every entry that is not excluded is about as likely as any other."""
    x, _ = G.make(3, V, dtype, 6, masked=0.0)
    x[0, ::3] = -INF
    x[1, 3:] = -INF
    x[2, V // 2:] = -INF
    y = torch.tensor([1, 2, 0])
    for k in (0, 5):
        _, got = G.run(lctx, x.repeat(times, 1), y.repeat(times), k, tau)
        want = in_fp32(R.stats(x, y, k, torch.tensor(tau).double()))
        G.compare(got, {n: v.repeat(times, *[1] * (v.dim() - 1)) for n, v in want.items()})


def rows_with_both_ends(V, dtype):
    dt = G.DT[dtype]
    most, low = torch.finfo(dt).max, torch.finfo(dt).min
    x, _ = G.make(7, V, dtype, 3, masked=0.0)
    x[0, 1], x[0, V - 1] = most, low                 # one certain token, one at the lowest value
    x[1] = low
    x[1, V // 2] = most                              # everything else at the lowest value
    x[2, ::2] = most
    x[2, 1::2] = low
    x[3, ::3] = -INF
    x[3, 1], x[3, 2] = most, low
    x[4, 0], x[4, V // 3], x[4, V - 2] = most / 2, -most / 2, low
    x[5] = low / 2
    x[5, 5] = most / 4
    x[6, V - 1] = most
    return x, torch.tensor([V - 1, 0, 1, 2, V // 3, 5, 0])


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("V,times", [(40, 1), (1003, 1), (1003, 300), (9000, 1), (20001, 1), (20001, 60), (33000, 60)])
@pytest.mark.parametrize("tau", [1.0, 0.7, 3.0, 2.0 ** 100, 2.0 ** 126])
def test_largest_and_lowest_value_in_one_row(lctx, V, times, dtype, tau):
    x, y = rows_with_both_ends(V, dtype)
    for k in (0, 6, 40):
        _, got = G.run(lctx, x.repeat(times, 1), y.repeat(times), k, tau)
        want = in_fp32(R.stats(x, y, k, torch.tensor(tau).double()))
        G.compare(got, {n: v.repeat(times, *[1] * (v.dim() - 1)) for n, v in want.items()})


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("tau", [1.0, 0.7, 2.0 ** 100, 2.0 ** 126, 2.0 ** -33])
def test_gradient_at_both_ends(lctx, dtype, tau):
    """Times the temperature, so that the step is 1."""
    x, y = rows_with_both_ends(1003, dtype)
    g = torch.Generator().manual_seed(5)
    ga, gb = torch.randn(7, generator=g), torch.randn(7, generator=g)
    G.check_grad(lctx, x, y, ga, None, tau, tau)
    if tau > 0.5:
        G.check_grad(lctx, x, y, ga, gb, tau, tau)
