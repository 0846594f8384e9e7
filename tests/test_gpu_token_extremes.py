"""Row statistics on the GPU at temperatures next to the limits, where products of logits leave fp32.  Results are those
of the fp64 statement, rounded to fp32 (a log-probability beyond it is -inf); tolerances are those of test_gpu_token.py."""
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
