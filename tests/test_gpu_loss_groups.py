"""The objectives where every CTA group takes several rows: the statistics, factors and teacher
entries of a row in flight beside those of its neighbours, shared-memory tiles used again, the
second and later exchanges of a cluster.  Compared with the definition in fp64 on the GPU.

A group takes rows r, r + groups, r + 2 groups, ...; a GB300 holds at most 912 groups of 64
threads, 608 of 128, 304 of 256, and fewer where a row takes a cluster of 2, 4 or 8 CTAs (152,
76, 38).  Every case has three to six rows per group.  Between valid rows there are ignored
ones: at random, the first of some groups, a run longer than a whole round of the groups, the
last ones.  They hold NaN.

Tolerances: REL and EPS of test_gpu_loss.py, whose derivation does not depend on the rows'
number (a thread adds at most 256 exponentials of a row in each of its chains).
"""
import pytest

torch = pytest.importorskip("torch")

import loss_scaled_adamw_gb300 as tl
from test_gpu_loss import DT, EPS, HALF_ULP, NAN, REL, TINY

pytestmark = pytest.mark.gpu
BLOCK = 1 << 24      # elements of an fp64 block


@pytest.fixture(scope="module")
def lctx():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from loss_scaled_adamw_gb300 import _build
    _build.build()
    return tl.tl_loss_create(8192, 64)


def logits(T, V, dtype, seed, groups):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = torch.randn(T, V, generator=g, device="cuda").mul_(3.0)
    y = torch.randint(0, V, (T,), generator=g, device="cuda")
    x[torch.arange(T, device="cuda"), y] += 5.0
    off = torch.rand(T, generator=g, device="cuda") < 0.25
    off[:5] = True
    off[groups + 9:2 * groups + 20] = True
    off[-3:] = True
    x[off] = NAN
    return g, x.to(DT[dtype]), torch.where(off, -100, y)


def blocks(T, V):
    n = max(1, BLOCK // V)
    return [(a, min(T, a + n)) for a in range(0, T, n)]


def near(got, want, tol, what):
    got, want = got.double(), want.double()
    bad = ~((got - want).abs() <= tol)
    assert not bool(bad.any()), (what, int(bad.sum()), bad.nonzero()[:4].tolist())


def near_gradient(got, want, dtype, band, listed, what):
    """band [T, 1]: the largest error at a listed element; others are within 2 REL of themselves."""
    tol = 4 * REL * want.abs() + band * listed
    tol = tol + (want.abs() + tol) * HALF_ULP[dtype] + TINY[dtype]
    near(got, want, tol, what)


def lp_of(x, y, tau):
    lp = torch.log_softmax(x.double() / tau, 1)
    return lp, lp.gather(1, y.clamp(min=0)[:, None])[:, 0]


# rows, vocabulary, type, groups at most (threads and CTAs of a group by tl's rules)
SHORT = (4200, 3001, "bf16", 912)          # 64 threads, a row in its tile
TILE = (3000, 6001, "bf16", 608)           # 128 threads, a row in its tile
STREAM = (2800, 16003, "f16", 608)         # 128 threads, a row over its tile: read again
STREAM32 = (2800, 12001, "f32", 608)
WIDE = (1300, 70001, "bf16", 304)          # 256 threads
PAIR = (700, 128256, "bf16", 152)          # clusters of 2 CTAs
QUAD = (360, 128256, "f32", 76)            # of 4
EIGHT = (170, 300001, "f32", 38)           # of 8


@pytest.mark.parametrize("shape,tau,ce,K,in_place", [
    (SHORT, 1.0, 0.0, 17, False), (SHORT, 3.0, 0.4, 100, True),
    (TILE, 2.0, 0.4, 64, False), (TILE, 1.0, 0.5, 300, True), (TILE, 4.0, 0.0, 5, False),
    (STREAM, 2.0, 0.25, 101, True), (STREAM, 0.7, 0.3, 33, False), (STREAM32, 1.0, 0.5, 300, False), (STREAM32, 1.0, 0.0, 3, True),
    (WIDE, 2.0, 0.25, 64, False), (PAIR, 2.0, 0.25, 64, True), (PAIR, 1.0, 0.0, 300, False), (QUAD, 3.0, 0.5, 64, False),
    (EIGHT, 1.0, 0.5, 20, True), (TILE, 1.0, 1.0, 0, False), (STREAM, 1.0, 1.0, 0, True), (PAIR, 1.0, 1.0, 0, True)])
def test_distillation(lctx, shape, tau, ce, K, in_place):
    """K = 0: the cross-entropy alone."""
    T, V, dtype, groups = shape
    g, x, y = logits(T, V, dtype, 50, groups)
    kd, n, scale = 0.75, 1000, 2.0 ** 8
    teacher = torch.randn(T, K, generator=g, device="cuda") * 3
    ids = torch.randint(0, V, (T, K), generator=g, device="cuda")
    if K:
        ids[:, ::7] = y.clamp(min=0)[:, None]              # the label, several times from 8 entries on
        ids[::3, K // 2:] = ids[::3, : K - K // 2]          # equal ids
        ids[1::5, -1] = -1                                  # padding
        ids[2::11] = -1                                     # no entries
        teacher[4::13, K // 3:] = -float("inf")
        teacher[y < 0] = NAN
        ids[y < 0] = V + 3
    listing = ids if in_place else ids.int()
    seed, loss, res = torch.tensor([scale], device="cuda"), torch.zeros(T, device="cuda"), torch.zeros(4, device="cuda")

    def call(v, out):
        tl.tl_distill_loss(lctx, v, teacher if K else None, listing if K else None, n, res, targets=y, kd_weight=kd,
                           ce_weight=ce, temperature=tau, seed=seed, dlogits=out, row_loss=loss)
        return out.clone(), loss.clone(), res.clone()

    first = call(x.clone(), torch.empty_like(x)) if not in_place else call(*[x.clone()] * 2)
    again = call(x.clone(), torch.empty_like(x)) if not in_place else call(*[x.clone()] * 2)
    assert all(torch.equal(a, b) for a, b in zip(first, again))
    dx, loss, res = first
    sums = torch.zeros(4, dtype=torch.float64, device="cuda")
    worst = 0.0
    for a, b in blocks(T, V):
        ok = (y[a:b] >= 0)
        x64 = torch.where(ok[:, None], x[a:b].double(), 0.0)
        want, listed = torch.zeros_like(x64), torch.zeros_like(x64)
        kds = ces = torch.zeros(b - a, dtype=torch.float64, device="cuda")
        kd_tol = torch.zeros_like(kds)
        if K:
            lq = torch.log_softmax(x64 / tau, 1)
            at = ids[a:b]
            use = (at >= 0) & ok[:, None]
            t = torch.where(use, teacher[a:b].double() / tau, -float("inf"))
            has = (t.amax(1) > -float("inf")).double()[:, None]
            lp = torch.log_softmax(t, 1)
            p = torch.where((t > -float("inf")), lp.exp(), 0.0)
            where = at.clamp(0, V - 1)
            lq_at = lq.gather(1, where)
            kds = tau * tau * torch.where(p > 0, p * (lp - lq_at), 0.0).sum(1)
            # differences of at most D, weights within 2 REL, two logarithms (test_gpu_loss_numbers.py)
            D = 2 * torch.where(p > 0, lq_at.abs(), 0.0).amax(1) + 2 * torch.where(p > 0, lp.abs(), 0.0).amax(1)
            kd_tol = tau * tau * ((2 * REL + 8 * EPS) * (D + 1) + 2 * REL)
            want += lq.exp() * (kd * tau * has)
            want.scatter_add_(1, where, -kd * tau * p)
            listed.scatter_(1, where, 1.0)
        if ce:
            l1, pick = lp_of(x64, y[a:b], 1.0)
            ces = -pick
            want += ce * l1.exp()
            where = y[a:b].clamp(min=0)[:, None]
            want.scatter_add_(1, where, torch.full_like(x64[:, :1], -ce))
            listed.scatter_(1, where, 1.0)
        row = ok * ((kd * kds if K else 0.0) + ce * ces)
        tol = ok * (kd * kd_tol + ce * (REL + 8 * EPS * ces.abs())) + 4 * EPS * row.abs()
        near(loss[a:b], row, tol, "loss")
        worst += float(tol.sum())
        sums += torch.stack([row.sum(), (ok * kds).sum(), (ok * ces).sum(), ok.sum().double()])
        want *= ok.double()[:, None] * (scale / n)
        near_gradient(dx[a:b], want, dtype, ok.double()[:, None] * (4 * REL * (kd * tau * (K > 0) + ce) * scale / n), listed, "dx")
    each = torch.tensor([1.0, 1.0 / kd, 1.0 / max(ce, 1e-3), 0.0], dtype=torch.float64, device="cuda") * worst
    div = torch.tensor([n, n, n, 1], dtype=torch.float64, device="cuda")
    near(res, sums / div, each / n + 4 * EPS * sums.abs() / div, "result")


@pytest.mark.parametrize("shape,tau,in_place", [
    (TILE, 1.0, False), (TILE, 0.7, True), (STREAM, 2.0, True), (STREAM32, 1.0, False), ((1300, 40003, "bf16", 304), 1.0, False),
    ((1300, 30002, "f32", 304), 0.7, True), (PAIR, 1.0, True), (QUAD, 1.0, False), (EIGHT, 1.0, True)])
def test_policy(lctx, shape, tau, in_place):
    T, V, dtype, groups = shape
    g, x, y = logits(T, V, dtype, 51, groups)
    n, scale, kl = 900, 2.0 ** 6, 0.05
    lp = torch.zeros(T, dtype=torch.float64, device="cuda")
    for a, b in blocks(T, V):
        lp[a:b] = torch.where(y[a:b] >= 0, lp_of(torch.nan_to_num(x[a:b]), y[a:b], tau)[1], 0.0)
    ok = y >= 0
    d = 0.3 * torch.randn(T, generator=g, device="cuda").double()
    for edge in (0.8, 1.2):           # no ratio so near the clip that rounding decides
        e = torch.tensor(edge, device="cuda").double().log()
        d = torch.where((d - e).abs() < 2e-3, d + 5e-3, d)
    old, ref = (lp - d).float(), (lp + 0.4 * torch.randn(T, generator=g, device="cuda").double()).float()
    adv = torch.randn(T, generator=g, device="cuda")
    for v in (old, ref, adv):
        v[~ok] = NAN
    seed, loss, got, res = (torch.zeros(k, device="cuda") for k in (1, T, T, 4))
    seed.fill_(scale)

    def call():
        v = x.clone()
        out = v if in_place else torch.empty_like(v)
        tl.tl_policy_loss(lctx, v, y, old, adv, n, res, ref_logp=ref, kl_weight=kl, temperature=tau, seed=seed, dlogits=out,
                          logp=got, row_loss=loss)
        return out, loss.clone(), got.clone(), res.clone()

    first, again = call(), call()
    assert all(torch.equal(a, b) for a, b in zip(first, again))
    dx, loss, got, res = first
    z = lambda v: torch.where(ok, v.double(), 0.0)  # noqa: E731
    A, r, b_ = z(adv), (lp - z(old)).exp(), z(ref) - lp
    free, held = r * A, r.clamp(0.8, 1.2) * A
    sur, k = -torch.minimum(free, held) * ok, (b_.exp() - b_ - 1) * ok
    grad = (torch.where(free <= held, -free, 0.0) + kl * (1 - b_.exp())) * ok
    e = (REL + 8 * EPS * lp.abs() + 2 * EPS * (lp.abs() + 1)) * ok
    size = r * A.abs() + kl * (b_.exp() + 1)
    tol = 2 * e * size + 4 * EPS * (size + A.abs() + 10 * kl)
    near(got, lp, e, "logp")
    near(loss, sur + kl * k, tol, "loss")
    sums = torch.stack([(sur + kl * k).sum() / n, sur.sum() / n, k.sum() / n, ok.sum().double()])
    kt = (2 * e * (b_.exp() + 1) + 4 * EPS * (b_.exp() + 10) * ok).sum() / n
    near(res, sums, torch.stack([tol.sum() / n, tol.sum() / n, kt, kt * 0]) + 4 * EPS * sums.abs(), "result")
    w = (grad * scale / n / tau)[:, None]
    wt = (tol * scale / n / tau)[:, None]          # the error of g: the terms of its loss
    for a, b in blocks(T, V):
        q = torch.log_softmax(torch.nan_to_num(x[a:b]).double() / tau, 1).exp()
        one = torch.zeros_like(q).scatter_(1, y[a:b].clamp(min=0)[:, None], 1.0)
        want = w[a:b] * (one - q)
        t = 4 * REL * want.abs() + wt[a:b] * (one + q) + (4 * REL * w[a:b].abs()) * one
        near(dx[a:b], want, t + (want.abs() + t) * HALF_ULP[dtype] + TINY[dtype], "dx")


@pytest.mark.parametrize("shape,pairs", [(TILE, 5), (STREAM, 40), (STREAM32, 1), (WIDE, 3), (PAIR, 8)])
def test_preference_and_log_probabilities(lctx, shape, pairs):
    """The statistics pass with its pairs' sums by the last group, and the gradient's own kernel."""
    T, V, dtype, groups = shape
    g, x, y = logits(T, V, dtype, 52, groups)
    ok, n, scale, beta = y >= 0, pairs, 2.0 ** 5, 0.02
    lp = torch.zeros(T, dtype=torch.float64, device="cuda")
    for a, b in blocks(T, V):
        lp[a:b] = torch.where(y[a:b] >= 0, lp_of(torch.nan_to_num(x[a:b]), y[a:b], 1.0)[1], 0.0)
    e = (REL + 8 * EPS * lp.abs()) * ok
    got = torch.zeros(T, device="cuda")
    tl.tl_token_logprob(lctx, x, y, got)
    near(got, lp, e, "token logp")
    ref = (lp + 0.4 * torch.randn(T, generator=g, device="cuda").double()).float()
    cut = torch.randperm(T - 2, generator=g, device="cuda")[: 2 * pairs + 1].sort().values + 1
    ratio = torch.where(ok, lp - ref.double(), 0.0)
    ref[~ok] = NAN
    seed = torch.tensor([scale], device="cuda")

    def call(in_place):
        v, o = x.clone(), [torch.zeros(k, device="cuda") for k in (T, pairs, 2 * pairs, 4)]
        out = v if in_place else torch.empty_like(v)
        tl.tl_preference_loss(lctx, v, y, cut, n, o[3], ref_logp=ref, beta=beta, seed=seed, dlogits=out, logp=o[0],
                              pair_loss=o[1], reward=o[2])
        return [out, *o]

    first, again = call(False), call(True)
    assert all(torch.equal(a, b) for a, b in zip(first, again))
    dx, got, loss, reward, res = first
    near(got, lp, e, "logp")
    bounds = cut.tolist()
    seqs = list(zip(bounds, bounds[1:]))
    want = beta * torch.stack([ratio[a:b].sum() for a, b in seqs])
    et = beta * torch.stack([(e + 4 * EPS)[a:b].sum() for a, b in seqs])
    near(reward, want, et + 4 * EPS * want.abs(), "reward")
    h, ht = want[0::2] - want[1::2], et[0::2] + et[1::2] + 4 * EPS * (want[0::2].abs() + want[1::2].abs() + 1)
    pair = torch.nn.functional.softplus(-h)
    near(loss, pair, ht + 4 * EPS * (1 + pair), "loss")
    near(res, torch.stack([pair.mean(), h.mean(), (h > 0).double().mean(), h.new_tensor(pairs)]),
         torch.stack([ht.mean() + 4 * EPS * (1 + pair.mean()), ht.mean(), h.new_tensor(EPS), h.new_tensor(0)]) + 4 * EPS, "result")
    down = torch.sigmoid(-h)
    gr = torch.zeros(T, dtype=torch.float64, device="cuda")
    gt = torch.zeros_like(gr)
    for i, (a, b) in enumerate(seqs):
        gr[a:b] = (beta if i % 2 else -beta) * down[i // 2]      # dL/dlp: negative in a chosen sequence
        gt[a:b] = beta * (ht[i // 2] + 8 * EPS) * down[i // 2]
    gr, gt = (gr * ok * scale / n)[:, None], (gt * ok * scale / n)[:, None]
    for a, b in blocks(T, V):
        q = torch.log_softmax(torch.nan_to_num(x[a:b]).double(), 1).exp()
        one = torch.zeros_like(q).scatter_(1, y[a:b].clamp(min=0)[:, None], 1.0)
        want = gr[a:b] * (one - q)
        t = 4 * REL * want.abs() + gt[a:b] * (one + q) + 4 * REL * gr[a:b].abs() * one
        near(dx[a:b], want, t + (want.abs() + t) * HALF_ULP[dtype] + TINY[dtype], "dx")


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
