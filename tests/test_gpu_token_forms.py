"""Row statistics on the GPU on either side of every rule that chooses how a row is held (its length, the number of
rows over the device's SMs), with fewer entries than alternatives among the rows.

Rows repeat a base of a few, so that the fp64 statement is taken once; tolerances are those of test_gpu_token.py."""
import pytest

torch = pytest.importorskip("torch")

import loss_scaled_adamw_gb300 as tl
import test_gpu_token as G
import token_reference as R

pytestmark = pytest.mark.gpu

lctx = G.lctx
INF = float("inf")


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def base_rows(V, dtype, seed):
    """Twelve rows: ordinary ones, and some with 0, 1, 5, 23 and 90 entries that are not excluded."""
    x, y = G.make(12, V, dtype, seed, masked=0.0)
    g = torch.Generator().manual_seed(seed)
    for row, n in ((1, 5), (2, 1), (4, 23), (5, 90), (7, 5), (8, 0), (10, 23)):
        keep = torch.randperm(V, generator=g)[:n]
        some = x[row, keep].clone()
        x[row] = -INF
        x[row, keep] = some
    y[3] = -100
    return x, y


def check_repeated(lctx, base, y0, rows, k, tau=1.0):
    """rows rows that follow the base in turns: all equal to the first ones bit for bit, those against the statement."""
    n = base.shape[0]
    x, y = base.cuda().repeat((rows + n - 1) // n, 1)[:rows], y0.cuda().repeat((rows + n - 1) // n)[:rows]
    f = lambda *s: torch.full(s, 7.0, device="cuda")  # noqa: E731
    out = {"logp": f(rows), "entropy": f(rows), "saved": f(rows, 3)}
    kw = {}
    if k:
        kw = dict(top_ids=torch.full((rows, k), 77, dtype=torch.int32, device="cuda"), top_logp=f(rows, k))
    tl.tl_token_stats(lctx, x, targets=y, temperature=tau, **out, **kw)
    out.update(ids=kw["top_ids"].long() if k else torch.empty(rows, 0).long().cuda(), top=kw["top_logp"] if k else f(rows, 0))
    for name, v in out.items():
        first = v[:n].repeat((rows + n - 1) // n, *[1] * (v.dim() - 1))[:rows]
        assert torch.equal(torch.nan_to_num(v, 1e9), torch.nan_to_num(first, 1e9)), name
    G.compare({name: v[:n].cpu() for name, v in out.items()}, R.stats(base, y0, k, tau))


@pytest.mark.parametrize("dtype,V", [("bf16", 6000), ("bf16", 12000), ("bf16", 2500), ("f16", 8192), ("f32", 3001)])
@pytest.mark.parametrize("k", [20, 100, 256])
def test_fewer_entries_than_alternatives_over_many_rows(lctx, dtype, V, k):
    """A team of warps goes from a row with few entries to the next without a barrier in the ordering of them: its count
    has to be the row's own in every warp, or places without an entry overwrite the entries."""
    base, y = base_rows(V, dtype, V + k)
    for _ in range(5):
        check_repeated(lctx, base, y, 40 * sms() + 5, k)
