"""The objectives where every CTA group takes several rows: sums over the launch's groups."""
import pytest

torch = pytest.importorskip("torch")

import loss_scaled_adamw_gb300 as tl
from test_gpu_loss import EPS

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lctx():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from loss_scaled_adamw_gb300 import _build
    _build.build()
    return tl.tl_loss_create(8192, 64)


def near(got, want, tol, what):
    got, want = got.double(), want.double()
    bad = ~((got - want).abs() <= tol)
    assert not bool(bad.any()), (what, int(bad.sum()), bad.nonzero()[:4].tolist())


@pytest.mark.parametrize("T,V", [(5000, 500), (5000, 4100), (1500, 30000)])
def test_sums_of_many_groups(lctx, T, V):
    """The mean terms are the fp64 sums of what the rows report, rounded once, call after call
    with other rows: the group that finishes last reads every group's slot, written by other CTAs."""
    g = torch.Generator(device="cuda")
    g.manual_seed(60)
    x = torch.randn(T, V, generator=g, device="cuda").bfloat16()
    y = torch.randint(-1, V, (T,), generator=g, device="cuda")
    old, adv = torch.full((T,), -9.0, device="cuda"), torch.randn(T, generator=g, device="cuda")
    loss, res = torch.zeros(40, T, device="cuda"), torch.zeros(40, 4, device="cuda")
    for i in range(40):
        tl.tl_policy_loss(lctx, x, y, old, adv * (i + 1), T, res[i], row_loss=loss[i])
    want = loss.double().sum(1) / T
    # fp64 sums differ in their order by far less than the fp32 result's own rounding
    near(res[:, 0], want, EPS * want.abs() + 1e-12 * loss.double().abs().sum(1), "loss")
    near(res[:, 1], want, EPS * want.abs() + 1e-12 * loss.double().abs().sum(1), "surrogate")
    assert bool((res[:, 3] == int((y >= 0).sum())).all())
