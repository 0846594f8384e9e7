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


def check_repeated(lctx, base, y0, rows, k, tau=1.0, pad=0):
    """rows rows that follow the base in turns, `pad` elements apart: all equal to the first ones bit for bit where they
    lie alike, and the first ones against the statement."""
    n = base.shape[0]
    x, y = base.cuda().repeat((rows + n - 1) // n, 1)[:rows], y0.cuda().repeat((rows + n - 1) // n)[:rows]
    if pad:
        x = torch.nn.functional.pad(x, (0, pad), value=12345.0)[:, :-pad]
    f = lambda *s: torch.full(s, 7.0, device="cuda")  # noqa: E731
    out = {"logp": f(rows), "entropy": f(rows), "saved": f(rows, 3)}
    kw = {}
    if k:
        kw = dict(top_ids=torch.full((rows, k), 77, dtype=torch.int32, device="cuda"), top_logp=f(rows, k))
    tl.tl_token_stats(lctx, x, targets=y, temperature=tau, **out, **kw)
    out.update(ids=kw["top_ids"].long() if k else torch.empty(rows, 0).long().cuda(), top=kw["top_logp"] if k else f(rows, 0))
    alike = (base.shape[1] + pad) * base.element_size() % 128 == 0   # else a row's phase says which threads sum what
    for name, v in out.items():
        if not alike and name != "ids":
            continue
        first = v[:n].repeat((rows + n - 1) // n, *[1] * (v.dim() - 1))[:rows]
        assert torch.equal(torch.nan_to_num(v, 1e9), torch.nan_to_num(first, 1e9)), name
    want = R.stats(base, y0, k, tau)
    for at in range(0, rows - n + 1, max(n, (rows // 8) // n * n)):   # stretches of the rows, from first to last
        G.compare({name: v[at:at + n].cpu() for name, v in out.items()}, want)


@pytest.mark.parametrize("dtype,V", [("bf16", 6000), ("bf16", 12000), ("bf16", 2500), ("f16", 8192), ("f32", 3001)])
@pytest.mark.parametrize("k", [20, 100, 256])
def test_fewer_entries_than_alternatives_over_many_rows(lctx, dtype, V, k):
    """A team of warps goes from a row with few entries to the next without a barrier in the ordering of them: its count
    has to be the row's own in every warp, or places without an entry overwrite the entries."""
    base, y = base_rows(V, dtype, V + k)
    for _ in range(5):
        check_repeated(lctx, base, y, 40 * sms() + 5, k)


# 16-bit and 32-bit lengths within each rule's range of 16-byte vectors: 257 to 512 and 513 to 1,024 of them in teams of
# one and two warps for many rows and of four for few; 2,049 to 4,096 in registers for few rows and streamed for many.
RANGES = {"one_warp_or_four": (4, {2: [2050, 3333, 4032], 4: [1100, 2001, 1984]}),
          "two_warps_or_four": (8, {2: [4500, 7001, 8128], 4: [2100, 4003, 4032]}),
          "registers_or_streamed": (2, {2: [16500, 30011, 32640], 4: [8300, 16001, 16320]})}


def tied_rows(V, dtype, seed):
    """Fourteen rows: the above, one of equal entries and one of three values (more candidates than a list holds)."""
    x, y = base_rows(V, dtype, seed)
    three = torch.randint(0, 3, (V,), generator=torch.Generator().manual_seed(seed)).to(x.dtype)
    return torch.cat([x, torch.full_like(x[:1], 0.75), three[None]]), torch.cat([y, torch.tensor([V - 1, 0])])


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rule", list(RANGES))
@pytest.mark.parametrize("k", [0, 8, 256])
def test_both_sides_of_the_rules_on_rows(lctx, rule, dtype, k):
    per_sm, lengths = RANGES[rule]
    for i, V in enumerate(lengths[4 if dtype == "f32" else 2]):
        base, y = tied_rows(V, dtype, V + k)
        for rows in (per_sm * sms(), per_sm * sms() + 1, 3 * per_sm * sms() + 7):
            check_repeated(lctx, base, y, rows, k, (1.0, 0.7)[i % 2], pad=(0, 3, 0)[i])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("k", [0, 33])
@pytest.mark.parametrize("V", [33001, 70016])
def test_rows_over_clusters_of_every_size(lctx, V, k, dtype):
    """Few long rows: eight, four, two and one CTA to a row."""
    base, y = tied_rows(V, dtype, V)
    for cluster in (8, 4, 2, 1):
        for rows in (sms() // cluster, sms() // cluster + 1):
            check_repeated(lctx, base, y, rows, k)
