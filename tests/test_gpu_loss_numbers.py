"""What the objectives' numbers promise beyond test_gpu_loss.py: a distillation loss made of
differences alone, rows without a softmax in distillation, the accuracy of a
log-probability, and arguments that are refused rather than dropped.

Constants of test_gpu_loss.py: EPS = 2^-24, REL bounds the relative error of an
exponential's share and the absolute one of the logarithm of a row's sum.
"""
import math

import pytest

torch = pytest.importorskip("torch")

import loss_reference as R
import loss_scaled_adamw_gb300 as tl
import test_gpu_loss as base
from test_gpu_loss import DT, EPS, INF, NAN, REL, close

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lctx():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from loss_scaled_adamw_gb300 import _build
    _build.build()
    return tl.tl_loss_create(20000, 64)


# --------------------------------------------------- distillation: differences alone

def kd_tolerance(x, teacher, ids, tau):
    """Per row, of kd = tau^2 (sum_i p_i (d_i / tau) + log p_r - log q_r), d_i = (t_i - t_r) -
    (x_i - x_r) against one reference entry r, the largest of the teacher's.  With D the
    largest |t_i - t_r| + |x_i - x_r|: a difference rounds three times, its product and the
    quotient by the sum once each (8 EPS D), and the weights p_i are within 2 REL; log p_r and
    log q_r are within REL and, through the scale of their exponent, 8 EPS of their own size."""
    tol = torch.zeros(x.shape[0], dtype=torch.float64)
    for t in range(x.shape[0]):
        at = [i for i, j in enumerate(ids[t].tolist()) if 0 <= j < x.shape[1] and teacher[t, i] > -INF]
        if not at:
            continue
        te, xe = teacher[t, at].double(), x[t, ids[t, at].long()].double()
        D = float(te.max() - te.min() + xe.max() - xe.min())
        log_q = (xe / tau - torch.logsumexp(x[t].double() / tau, 0)).abs().max()
        log_p = math.log(len(at))
        tol[t] = tau * (2 * REL + 8 * EPS) * D + tau * tau * (2 * REL + 8 * EPS * (log_p + float(log_q)))
    return tol


@pytest.mark.parametrize("tau", [0.1, 0.7, 1.0, 2.0, 3.0])
@pytest.mark.parametrize("V,K", [(300, 6), (9000, 40), (9000, 300), (70000, 17)])
def test_distillation_is_the_same_at_any_offset(lctx, V, K, tau):
    """A common offset of a row's logits, of the student or the teacher, changes nothing, nor do
    finite masks of -1e9 and -1e30 all over a row: the loss is a function of differences.
    Logits are multiples of 1/64 below 2^18 (of 64 at 1e9), so every difference is exact."""
    g, x, y = base.make(10, V, "f32", 30, masked=0.0)
    x = (x * 64).round() / 64
    teacher, ids = base.teacher_of(10, V, K, g)
    teacher = (teacher * 64).round() / 64
    for t, (student, other) in enumerate([(0.0, 0.0), (1e3, 0.0), (-3e4, 5e4), (1.8e5, -2.0 ** 17), (-2.0 ** 17, 1.0),
                                          (0.0, 2.0 ** 17)]):
        x[t] += student
        teacher[t] += other
    x[6] = -1e9
    x[6, ids[6, :3].long()] = torch.tensor([-1e9 + 128, -1e9 + 64, -1e9])   # fp32 spacing there is 64
    y[6] = ids[6, 0]
    x[7], teacher[7] = -1e30, -1e30
    teacher[8] = -1e9
    x[9, : V // 2] = -1e9
    ids[9] = V // 2 + ids[9] % (V - V // 2)
    y[9] = V - 1
    # the statement gets the teacher's differences: a log-sum at -1e30 would lose log K in 64 bits too
    from_top = teacher.double() - teacher.double().amax(1, keepdim=True)
    for kd, ce in ((1.0, 0.0), (0.5, 0.5)):
        got = base.run_distill(lctx, x, teacher, ids, 10, y, kd, ce, tau, backward=False)
        want = R.distill(x, from_top, ids, 10, y, kd, ce, tau)
        kd_tol = kd_tolerance(x, teacher, ids, tau)
        ce_row = (want["loss"] - kd * want["kd"]) / ce if ce else torch.zeros(10, dtype=torch.float64)
        ce_tol = REL + 8 * EPS * ce_row.abs()
        tol = kd * kd_tol + ce * ce_tol + 4 * EPS * want["loss"].abs()
        close(got["loss"], want["loss"], tol, "loss")
        r = want["result"].double()
        st = torch.stack([tol.sum() / 10, kd_tol.sum() / 10, ce_tol.sum() / 10 * (ce > 0), torch.tensor(0.0).double()])
        close(got["result"], r, st + 4 * EPS * r.abs(), "result")


# ------------------------------------------------- distillation: rows without a softmax

@pytest.mark.parametrize("V", [40, 700, 9000, 70000])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("tau", [1.0, 2.0, 3.0])
def test_distillation_of_rows_without_a_softmax(lctx, V, dtype, tau):
    """A valid row with a NaN or +inf logit, with nothing but -inf, or with a teacher entry of
    NaN or +inf is NaN in its loss and in its whole gradient, whatever the teacher lists and
    whatever the weights; the rows beside it are not."""
    T, K = 16, 5
    g, x, y = base.make(T, V, dtype, 31, masked=0.0)
    teacher, ids = base.teacher_of(T, V, K, g)
    for t in range(0, 9):                    # NaN, +inf, -inf: with entries, padded ones, -inf ones
        x[t, V // 3] = (NAN, INF, 0.0)[t % 3]
        if t % 3 == 2:
            x[t] = -INF
        if t in (3, 4, 5):
            ids[t] = -1
        if t in (6, 7, 8):
            teacher[t] = -INF
    teacher[9, 2], teacher[10, 4] = NAN, INF
    ids[11] = -1                              # no entries: kd = 0
    teacher[12] = -INF                        # the same
    bad = torch.zeros(T, dtype=torch.bool)
    for kd, ce, k in ((1.0, 0.0, K), (0.6, 0.4, K), (0.6, 0.0, 0), (0.6, 0.4, 0), (0.0, 0.0, K)):
        bad[:9], bad[9:11] = True, k > 0 and kd > 0
        te, ti = (teacher, ids) if k else (None, None)
        for in_place in (False, True):
            got = base.run_distill(lctx, x, te, ti, T, y, kd, ce, tau, 4.0, in_place=in_place)
            dx = torch.isnan(got["dx"].float())
            assert torch.equal(torch.isnan(got["loss"]).cpu(), bad), (kd, ce, k)
            assert torch.equal(dx.all(1).cpu(), bad) and torch.equal(dx.any(1).cpu(), bad), (kd, ce, k)
            assert math.isnan(float(got["result"][0])) and float(got["result"][3]) == T
            # the others are what they are without the bad rows beside them
            ok = ~bad
            want = R.distill(x[ok], te[ok] if k else None, ti[ok] if k else None, T, y[ok], kd, ce, tau, 4.0)
            w = torch.full((int(ok.sum()),), 4.0 / T * (kd * tau + ce), dtype=torch.float64)
            hot = base.hot(y[ok], V)
            if k:
                for i, row in enumerate(ti[ok].tolist()):
                    for j in row:
                        if j >= 0:
                            hot[i, j] = True
            base.check_dx(got["dx"][ok.cuda()], want["dx"], dtype, w, torch.full_like(w, 2 * REL + 64 * EPS), hot, "dx")


# ------------------------------------------------------------ accuracy of log-probabilities

def scored(T, V, dtype, seed, spread=2.5):
    """Logits on the GPU, random labels, and the labels' log-probabilities in 64 bits."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = (torch.randn(T, V, generator=g, device="cuda") * spread).to(DT[dtype])
    y = torch.randint(0, V, (T,), generator=g, device="cuda")
    want = torch.cat([torch.log_softmax(x[a:a + 256].double(), 1).gather(1, y[a:a + 256, None])[:, 0]
                      for a in range(0, T, 256)])
    return g, x, y, want


def with_three_roundings(x, y):
    """log q_y formed as ((x_y log2 e - u - n) - log2 of the sum's rest) ln 2 in fp32, each step
    rounded, from a sum that is exact: what the kernel would give if it did not carry errors along."""
    f = lambda v: v.float().double()  # noqa: E731
    c, ln2 = torch.tensor(1.4426950408889634).double(), torch.tensor(0.6931471805599453).double()
    out = []
    for a in range(0, x.shape[0], 256):
        z = x[a:a + 256].double()
        u = torch.round(z.amax(1) * c)
        s = f(torch.exp2(z * c - u[:, None]).sum(1))
        n = torch.floor(torch.log2(s))
        rest = f(torch.log2(s * torch.exp2(-n)))
        p = f(z.gather(1, y[a:a + 256, None])[:, 0] * c - (u + n))
        out.append(f(f(p - rest) * ln2))
    return torch.cat(out)


@pytest.mark.parametrize("T,V,dtype", [(4096, 8192, "f32"), (4096, 1000, "f16"), (2048, 50001, "bf16"), (1024, 128256, "bf16")])
def test_log_probabilities_are_rounded_once(lctx, T, V, dtype):
    """Over many rows (temperature 1).  Rounding the result itself has the rms q of the exact
    values.  The logarithm of the sum adds: an exponential's error of at most 2^-22, as if one
    term made the sum and the error were uniform (1.4e-7); the roundings of partial sums, eight
    or so on the way of a term that counts, 0.35e-7 each (1e-7); log2's last place (0.4e-7):
    1.8e-7, taken as 2e-7.  The scale log2 e is off by 1.34e-8 of itself in fp32, which moves
    every result by that part of x_y - E_q[x], in the mean the logits' variance 6.25: 0.84e-7;
    with a mean error of the exponential within 2^-24 the mean is held to 1.5e-7 + 5 rms /
    sqrt(T), and the rms is taken about the mean.  An rms of T rows strays by 5 / sqrt(2 T)."""
    g, x, y, want = scored(T, V, dtype, 40)
    lp = torch.zeros(T, device="cuda")
    tl.tl_token_logprob(lctx, x, y, lp)
    q = float((want.float().double() - want).square().mean().sqrt())
    bound = math.sqrt(q * q + 2e-7 ** 2) * (1 + 5 / math.sqrt(2 * T))
    rms = lambda e: float((e - e.mean()).square().mean().sqrt())  # noqa: E731
    e = lp.double() - want
    assert rms(with_three_roundings(x, y) - want) > bound        # the bound tells them apart
    assert rms(e) <= bound, (rms(e), bound)
    assert abs(float(e.mean())) <= 1.5e-7 + 5 * bound / math.sqrt(T), float(e.mean())


@pytest.mark.parametrize("V,dtype", [(126599, "f32"), (128256, "bf16")])
@pytest.mark.parametrize("tau", [0.7, 0.5])
def test_small_terms_of_a_long_row_are_not_lost(lctx, V, dtype, tau):
    """Below 1 a temperature spreads a row's exponentials over tens of bits, and most of them are
    small against a thread's sum: added one at a time, more of them fall below half of its last
    place than round up, and every log-probability comes out high (by 1.5e-7 and 2.4e-7 for these
    two, from additions in fp32 alone).  The mean is held to the exponential's mean error (2^-24) and five
    standard errors; per row an exponent of up to 32 bits rounds by up to 2^-20 (rms
    3.8e-7 in the sum where one term makes it), beside the result's rounding q: with 5e-7 for
    all but q.  The definition is taken at the scale that the kernel has, 1 / tau times log2 e in fp32."""
    T = 4096
    g = torch.Generator(device="cuda")
    g.manual_seed(42)
    x = (torch.randn(T, V, generator=g, device="cuda") * 2.5)
    y = torch.randint(0, V, (T,), generator=g, device="cuda")
    x[torch.arange(T, device="cuda"), y] += 2 + 12 * torch.rand(T, generator=g, device="cuda")
    x = x.to(DT[dtype])
    f = lambda v: torch.tensor(v, dtype=torch.float32)  # noqa: E731
    scale = float((f(1.0) / f(tau)) * f(1.4426950408889634)) * math.log(2.0)
    want = torch.cat([torch.log_softmax(x[a:a + 64].double() * scale, 1).gather(1, y[a:a + 64, None])[:, 0]
                      for a in range(0, T, 64)])
    lp = torch.zeros(T, device="cuda")
    tl.tl_token_logprob(lctx, x, y, lp, temperature=tau)
    q2 = float((want.float().double() - want).square().mean())
    assert abs(float((lp.double() - want).mean())) <= 2.0 ** -24 + 5 * math.sqrt(q2 + 5e-7 ** 2) / math.sqrt(T)


def test_rewards_of_long_sequences(lctx):
    """beta times a sum of 4,000 rows' lp - ref.  Per row the errors of the test above, rms 3.5e-7
    and mean 1.5e-7; lp - ref (at most 2) rounds by 1.2e-7 more, unbiased."""
    T, V, L = 8192, 2000, 4000
    g, x, y, want = scored(T, V, "f32", 41)
    ref = (want + 0.3 * torch.randn(T, generator=g, device="cuda").double()).float()
    seq = torch.tensor([7, 7 + L, 7 + 2 * L], device="cuda")
    res, rew = torch.zeros(4, device="cuda"), torch.zeros(2, device="cuda")
    tl.tl_preference_loss(lctx, x, y, seq, 1, res, ref_logp=ref, beta=0.1, reward=rew)
    d = want - ref.double()
    exact = 0.1 * torch.stack([d[7:7 + L].sum(), d[7 + L:7 + 2 * L].sum()])
    tol = 0.1 * (5 * math.sqrt(3.5e-7 ** 2 + 1.2e-7 ** 2) * math.sqrt(L) + 1.5e-7 * L) + 4 * EPS * exact.abs().cpu()
    close(rew, exact.cpu(), tol, "reward")


# --------------------------------------------------------- rows outside every sequence

def test_rows_outside_every_sequence(lctx):
    """They are in no sum and have a zero gradient, NaN logits or not; their logp is what it is."""
    T, V, seq = 12, 700, [2, 5, 7, 7, 10]
    g, x, y = base.make(T, V, "f32", 33, masked=0.0)
    x[11, 3] = NAN
    got = base.run_preference(lctx, x, y, seq, 2, seed=4.0)
    sane = torch.nan_to_num(x)
    want = R.preference(sane, y, seq, 2, seed=4.0)
    want["logp"][11] = NAN
    base.check_preference(got, want, sane, y, seq, 2, "f32", 0.1, 1.0, 4.0, None)
    assert float(got["dx"][[0, 1, 10, 11]].abs().max()) == 0.0


# ------------------------------------------------------------------------- refusals

def test_nothing_that_is_given_is_dropped(lctx):
    T, V = 4, 64
    x, y = torch.zeros(T, V, device="cuda"), torch.zeros(T, dtype=torch.int64, device="cuda")
    ids, tea = torch.zeros(T, 2, dtype=torch.int32, device="cuda"), torch.zeros(T, 2, device="cuda")
    f, res = torch.zeros(T, device="cuda"), torch.zeros(4, device="cuda")
    before = tl.tl_loss_launch_count(lctx)
    for call in (lambda: tl.tl_distill_loss(lctx, x, None, ids, 4, res, targets=y, ce_weight=1.0),
                 lambda: tl.tl_distill_loss(lctx, x, tea, None, 4, res, targets=y, ce_weight=1.0),
                 lambda: tl.tl_policy_loss(lctx, x, y, f, f, 4, res, seed=0),       # the scale of a destroyed context
                 lambda: tl.tl_preference_loss(lctx, x, y, torch.tensor([0, 2, 4], device="cuda"), 1, res, seed=0),
                 lambda: tl.tl_distill_loss(lctx, x, tea, ids, 4, res, seed=0)):
        with pytest.raises(ValueError):
            call()
    assert tl.tl_loss_launch_count(lctx) == before
