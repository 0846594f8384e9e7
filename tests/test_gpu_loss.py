"""The objectives over logits on the GPU against their fp64 statements (loss_reference.py).

Tolerances, derived from the arithmetic (eps = 2^-24, the unit roundoff of fp32):
* e_j = exp((x_j - M) it): the subtraction, the product and the constant each round once,
  so the exponent a (in bits) is off by 3 eps |a|; the terms that carry a row's sum have
  |a| <= 30: 0.69 * 3 * 30 eps = 3.7e-6, and the exponential itself adds 2^-22.  A row sum
  adds positive terms in chains of at most 256 (a thread's elements, then a tree):
  256 eps = 1.5e-5.  Together REL = 2.5e-5 bounds the relative error of S, of q for such
  terms, and the absolute one of log S; smaller q (|a| up to 130) are within 2 REL.
* lp = (x_y - M) it - log S: REL + 4 eps |lp|.
* policy: r = exp(lp - old) is off by the error of lp; KL's exp(d) alike, and its
  difference exp(d) - d - 1 by eps (|e^d| + |d|) more.
* preference: h is beta times a sum of at most L rows' lp: beta L (REL + 4 eps max|lp|);
  sg and log sg have derivatives of at most 1 in h.
* distill: a mean over p of logits' differences: REL plus 8 eps of the largest magnitude
  entering it, times tau^2.
* a gradient w (1[j = y] - q_j): |w| (rel(w) + 2 REL) q, plus |w| (rel(w) + 2 REL) at
  listed entries, rounded once to the type (half an ulp; fp16 subnormals 2^-25).  An
  exponential below 2^-126 is taken as 0: |w| 2^-126.
"""
import math

import pytest

torch = pytest.importorskip("torch")

import loss_reference as R
import loss_scaled_adamw_gb300 as tl

pytestmark = pytest.mark.gpu

EPS, REL = 2.0 ** -24, 2.5e-5
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
HALF_ULP = {k: torch.finfo(v).eps / 2 for k, v in DT.items()}
TINY = {"bf16": 1e-38, "f16": 2.0 ** -24, "f32": 1e-38}
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lctx():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from loss_scaled_adamw_gb300 import _build
    _build.build()
    return tl.tl_loss_create(20000, 64)


class Rows:
    """A [T, V] device matrix inside a canary-filled buffer: `pad` extra elements between
    rows and `lead` before the first."""

    def __init__(self, T, V, dtype, pad=0, lead=0, values=None):
        self.ld, self.T, self.V, self.lead = V + pad, T, V, lead
        self.buf = torch.full((lead + T * self.ld + 64,), 12345.0, dtype=dtype, device="cuda")
        self.t = self.buf[lead:lead + T * self.ld].view(T, self.ld)[:, :V]
        if values is not None:
            self.t.copy_(values)

    def outside_untouched(self):
        mask = torch.ones_like(self.buf, dtype=torch.bool)
        mask[self.lead:self.lead + self.T * self.ld].view(self.T, self.ld)[:, :self.V] = False
        return bool((self.buf[mask] == 12345.0).all())


def make(T, V, dtype, seed, masked=0.25, spread=3.0):
    g = torch.Generator().manual_seed(1000 * seed + 7 * T + V)
    x = torch.randn(T, V, generator=g) * spread
    y = torch.randint(0, V, (T,), generator=g)
    for t in range(T):
        x[t, y[t]] += 4.0
    if T > 1:
        y = torch.where(torch.rand(T, generator=g) < masked, -100, y)
    return g, x.to(DT[dtype]), y


def close(got, want, tol, what):
    got, want = got.detach().cpu().double().reshape(-1), want.double().reshape(-1)
    tol = torch.as_tensor(tol, dtype=torch.float64).expand_as(want) if not isinstance(tol, torch.Tensor) else tol.reshape(-1)
    assert torch.equal(torch.isnan(got), torch.isnan(want)), what
    inf = torch.isinf(want)
    assert torch.equal(got[inf], want[inf]), what
    ok = ~torch.isnan(want) & ~inf
    bad = (got[ok] - want[ok]).abs() > tol[ok]
    assert not bool(bad.any()), (what, int(bad.sum()), float(((got[ok] - want[ok]).abs() / tol[ok]).max()))


def lp_tol(lp):
    return REL + 4 * EPS * torch.nan_to_num(lp.abs(), nan=0.0, posinf=0.0, neginf=0.0)


def check_dx(got, want, dtype, w, rel_w, entries, what):
    """w: bound of |w| per row; rel_w: its relative error; entries: bool [T, V], listed positions."""
    band = (w * (rel_w + 2 * REL))[:, None]
    tol = (2 * REL + rel_w)[:, None] * want.abs() + band * entries.double()
    tol = tol + (want.abs() + tol) * HALF_ULP[dtype] + TINY[dtype] + (w * 2.0 ** -126)[:, None]
    close(got.float(), want, torch.nan_to_num(tol, nan=0.0, posinf=0.0), what)


def hot(y, V):
    m = torch.zeros(y.shape[0], V, dtype=torch.bool)
    for t, j in enumerate(y.tolist()):
        if 0 <= j < V:
            m[t, j] = True
    return m


def cu(t):
    return None if t is None else t.cuda()


# --------------------------------------------------------------------- calls

def run_policy(lctx, x, y, old, adv, n, ref=None, kl=0.0, tau=1.0, seed=None, pad=0, lead=0, dpad=None, dlead=None,
               in_place=False, backward=True, clip=(0.2, 0.2)):
    T, V = x.shape
    X = Rows(T, V, x.dtype, pad, lead, x.cuda())
    D = X if in_place else Rows(T, V, x.dtype, pad if dpad is None else dpad, lead if dlead is None else dlead)
    lp, loss, res = (torch.full((k,), 77.0, device="cuda") for k in (T, T, 4))
    s = None if seed is None else torch.tensor([seed], device="cuda")
    tl.tl_policy_loss(lctx, X.t, cu(y), cu(old), cu(adv), n, res, ref_logp=cu(ref), clip_low=clip[0], clip_high=clip[1],
                      kl_weight=kl, temperature=tau, seed=s, dlogits=D.t if backward else None, logp=lp, row_loss=loss)
    torch.cuda.synchronize()
    assert X.outside_untouched() and D.outside_untouched()
    if not in_place:
        assert torch.equal(X.t.cpu().view(torch.int16 if x.dtype != torch.float32 else torch.int32),
                           x.view(torch.int16 if x.dtype != torch.float32 else torch.int32))
    return {"logp": lp, "loss": loss, "result": res, "dx": D.t}


def check_policy(got, ref, x, y, old, adv, n, dtype, tau, seed, kl, rl, backward=True):
    V = x.shape[1]
    close(got["logp"], ref["logp"], lp_tol(ref["logp"]), "logp")
    lp = torch.nan_to_num(ref["logp"])
    e = lp_tol(lp) + 2 * EPS * (lp.abs() + 1)
    r = torch.exp(lp - torch.nan_to_num(old.double()))
    k = torch.exp((torch.nan_to_num(rl.double()) - lp) if rl is not None else torch.zeros_like(lp))
    A = torch.nan_to_num(adv.double()).abs()
    tol = 2 * e * (r * A + kl * (k + 1)) + 4 * EPS * (A * (r + 1) + kl * (k + 10))
    tol = torch.where(y >= 0, tol, 0.0)
    close(got["loss"], ref["loss"], tol, "loss")
    kt = torch.where(y >= 0, 2 * e * (k + 1) + 4 * EPS * (k + 10), 0.0)
    want = ref["result"].double()
    st = torch.stack([tol.sum() / n, tol.sum() / n, kt.sum() / n, torch.tensor(0.0).double()])
    close(got["result"], want, st + 2 * EPS * want.abs(), "result")
    if backward:
        w = torch.nan_to_num((r * A + kl * (k + 1)) * seed / n / tau)
        gw = torch.nan_to_num(ref["g"].abs()) * seed / n / tau
        # the error of g relative to its own size (the KL term may cancel the surrogate)
        rel = torch.where(gw > 0, torch.minimum(2 * e * w / gw + 4 * EPS * w / gw + 8 * EPS, torch.tensor(1e9).double()), 0.0)
        check_dx(got["dx"], ref["dx"], dtype, gw, rel, hot(y, V), "dx")


@pytest.mark.parametrize("V", [1, 2, 7, 33, 127, 1000, 1025, 4097, 8192, 32003, 50001])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_policy_over_vocabularies(lctx, V, dtype):
    T = 6 if V > 5000 else 13
    g, x, y = make(T, V, dtype, 1)
    tau, kl, seed = (0.7, 0.05, 2.0 ** 10)
    lp = R.logprob(x, y, tau)
    old = (lp + 0.3 * torch.randn(T, generator=g)).float()
    adv, ref = torch.randn(T, generator=g), (lp + 0.5 * torch.randn(T, generator=g)).float()
    old[y < 0], adv[y < 0], ref[y < 0] = NAN, NAN, INF
    got = run_policy(lctx, x, y, old, adv, 5, ref, kl, tau, seed, pad=3, lead=1)
    want = R.policy(x, y, old, adv, 5, ref, kl_weight=kl, tau=tau, seed=seed)
    check_policy(got, want, x, y, old, adv, 5, dtype, tau, seed, kl, ref)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [128256, 300001])
def test_policy_large_vocabulary(lctx, V, dtype):
    T = 3
    g, x, y = make(T, V, dtype, 2, masked=0.0)
    lp = R.logprob(x, y)
    old, adv = (lp + 0.2).float(), torch.tensor([-1.0, 2.0, -0.5])
    got = run_policy(lctx, x, y, old, adv, 3, None, 0.0, 1.0, 1.0)
    check_policy(got, R.policy(x, y, old, adv, 3), x, y, old, adv, 3, dtype, 1.0, 1.0, 0.0, None)


@pytest.mark.parametrize("layout", [dict(pad=0, lead=0), dict(pad=5, lead=3), dict(pad=8, lead=8),
                                    dict(pad=0, lead=0, dpad=3, dlead=1), dict(pad=1, lead=2, in_place=True),
                                    dict(pad=0, lead=0, in_place=True), dict(pad=24, lead=4, dpad=40, dlead=4),
                                    dict(pad=0, lead=0, backward=False)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_policy_layouts(lctx, layout, dtype):
    T, V = 9, 3001
    g, x, y = make(T, V, dtype, 3)
    lp = R.logprob(x, y)
    old, adv = (lp + 0.3 * torch.randn(T, generator=g)).float(), torch.randn(T, generator=g)
    got = run_policy(lctx, x, y, old, adv, 7, seed=4.0, **layout)
    check_policy(got, R.policy(x, y, old, adv, 7, seed=4.0), x, y, old, adv, 7, dtype, 1.0, 4.0, 0.0, None,
                 layout.get("backward", True))


@pytest.mark.parametrize("T", [0, 1, 2, 151, 700])
def test_policy_row_counts(lctx, T):
    V = 257
    g, x, y = make(T, V, "f16", 4)
    lp = R.logprob(x, y)
    old, adv = (lp + 0.3 * torch.randn(T, generator=g)).float(), torch.randn(T, generator=g)
    got = run_policy(lctx, x, y, old, adv, max(1, T), seed=8.0)
    check_policy(got, R.policy(x, y, old, adv, max(1, T), seed=8.0), x, y, old, adv, max(1, T), "f16", 1.0, 8.0, 0.0, None)


@pytest.mark.parametrize("V", [40, 8192, 128256])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_rows_with_masks_and_non_finite_logits(lctx, V, dtype):
    """Excluded tokens (-inf, the type's lowest value), rows without a softmax, targets beyond
    the vocabulary, ignored rows full of NaN: each row stands for itself."""
    T = 9
    g, x, y = make(T, V, dtype, 5, masked=0.0)
    low = torch.finfo(DT[dtype]).min
    x[0, ::2] = -INF; y[0] = 1                   # half the vocabulary excluded
    x[1, :] = -INF; x[1, 3] = 0.5; y[1] = 3        # one token left: lp = 0, gradient 0
    x[2, :] = low                                # all at the lowest value: uniform
    x[3, :] = low; x[3, 5] = 0.0; y[3] = 5
    x[4, :] = -INF                               # nothing left
    x[5, 7] = INF
    x[6, V - 1] = NAN
    y[7] = V                                     # not an id
    x[8, :] = NAN; y[8] = -1                     # ignored
    lp = R.logprob(x, y)
    old = torch.nan_to_num(lp).float() + 0.1
    adv = torch.ones(T)
    for in_place in (False, True):
        got = run_policy(lctx, x, y, old, adv, 8, seed=2.0, in_place=in_place)
        want = R.policy(x, y, old, adv, 8, seed=2.0)
        check_policy(got, want, x, y, old, adv, 8, dtype, 1.0, 2.0, 0.0, None)
        nan_rows = torch.isnan(got["dx"].float()).all(1).cpu()
        assert nan_rows.tolist() == [False] * 4 + [True] * 4 + [False]
        assert math.isnan(float(got["result"][0])) and float(got["result"][3]) == 8
    x[1, 3], y[1] = -INF, 4                      # excluded target: lp = -inf, ratio 0
    x[1, 4:6] = torch.tensor([-INF, 1.0])
    lp = torch.zeros(T)
    lp_gpu = lp.cuda()
    tl.tl_token_logprob(lctx, x.cuda(), y.cuda(), lp_gpu)
    assert float(lp_gpu[1]) == -INF and float(lp_gpu[8]) == 0.0


@pytest.mark.parametrize("tau", [1.0, 0.1, 2.0, 1e-4, 1e30])
@pytest.mark.parametrize("V", [300, 9000, 70000])
def test_logits_of_any_magnitude(lctx, V, tau):
    """Logits far from zero (a common offset, finite masks of -1e9 and the like, in part of a
    row and all over it), and temperatures far from 1: only differences count.  The offsets
    are multiples of what keeps x itself exact; each fp32 difference is then exact too."""
    g, x, y = make(8, V, "f32", 20, masked=0.0)
    x = (x * 64).round() / 64                                   # 1/64 steps: exact below 2^18
    for t, off in enumerate([0.0, 1e3, -3e4, 7.2e5 / 4, -2.0 ** 17, 0.0, 0.0, 0.0]):
        x[t] += off
    x[5, : V // 2] = -1e9
    x[6] = -1e9
    x[6, 3:6] = torch.tensor([-1e9 + 128, -1e9 + 64, -1e9])    # spacing of fp32 there
    x[7] = -1e30
    y[5], y[6] = V - 1, 3
    lp = R.logprob(x, y, tau)
    old, adv = torch.where(torch.isfinite(lp), lp, 0.0).float(), torch.ones(8)
    got = run_policy(lctx, x, y, old, adv, 8, tau=tau, seed=4.0)
    want = R.policy(x, y, old, adv, 8, tau=tau, seed=4.0)
    check_policy(got, want, x, y, old, adv, 8, "f32", tau, 4.0, 0.0, None)
    teacher, ids = teacher_of(8, V, 6, g)
    if tau in (0.1, 1.0, 2.0):
        got = run_distill(lctx, x, teacher, ids, 8, y, 0.5, 0.5, tau, 1.0)
        want = R.distill(x, teacher, ids, 8, y, 0.5, 0.5, tau, 1.0)
        listed = hot(y, V)
        for t in range(8):
            listed[t, ids[t].long()] = True
        w = torch.full((8,), (0.5 * tau + 0.5) / 8, dtype=torch.float64)
        check_dx(got["dx"], want["dx"], "f32", w, torch.full((8,), 2 * REL + 64 * EPS, dtype=torch.float64), listed, "dx")


def test_all_rows_ignored_give_zeros(lctx):
    x = torch.full((5, 1000), NAN, dtype=torch.bfloat16)
    y = torch.full((5,), -100)
    got = run_policy(lctx, x, y, torch.full((5,), NAN), torch.full((5,), NAN), 1)
    assert float(got["dx"].float().abs().max()) == 0.0
    assert got["result"].tolist() == [0.0, 0.0, 0.0, 0.0] and got["logp"].tolist() == [0.0] * 5


@pytest.mark.parametrize("T,V,dtype,tau", [(1, 128256, "bf16", 1.0), (1, 5, "f32", 1.0), (4, 50001, "f16", 0.7),
                                           (300, 513, "bf16", 2.0), (2, 300001, "f32", 1.0), (37, 8192, "f32", 1.3)])
def test_token_logprob(lctx, T, V, dtype, tau):
    g, x, y = make(T, V, dtype, 6)
    X = Rows(T, V, DT[dtype], 1, 1, x.cuda())
    lp = torch.full((T,), 9.0, device="cuda")
    tl.tl_token_logprob(lctx, X.t, y.cuda(), lp, temperature=tau)
    want = R.logprob(x, y, tau)
    close(lp, want, lp_tol(want), "logp")
    assert X.outside_untouched()


# ------------------------------------------------------------------ preference

def run_preference(lctx, x, y, seq, n, ref=None, beta=0.1, smooth=0.0, tau=1.0, seed=None, pad=0, lead=0,
                   in_place=False, backward=True):
    T, V = x.shape
    X = Rows(T, V, x.dtype, pad, lead, x.cuda())
    D = X if in_place else Rows(T, V, x.dtype, pad, lead)
    P = len(seq) // 2
    lp, loss, rew, res = (torch.full((k,), 77.0, device="cuda") for k in (T, P, 2 * P, 4))
    s = None if seed is None else torch.tensor([seed], device="cuda")
    tl.tl_preference_loss(lctx, X.t, cu(y), torch.tensor(seq, device="cuda"), n, res, ref_logp=cu(ref), beta=beta,
                          label_smoothing=smooth, temperature=tau, seed=s, dlogits=D.t if backward else None, logp=lp,
                          pair_loss=loss, reward=rew)
    torch.cuda.synchronize()
    assert X.outside_untouched() and D.outside_untouched()
    return {"logp": lp, "loss": loss, "reward": rew, "result": res, "dx": D.t}


def check_preference(got, want, x, y, seq, n, dtype, beta, tau, seed, ref, backward=True):
    T, V = x.shape
    close(got["logp"], want["logp"], lp_tol(want["logp"]), "logp")
    e = torch.where(y >= 0, lp_tol(want["logp"]) + 2 * EPS * (0 if ref is None else torch.nan_to_num(ref.double().abs())), 0.0)
    s = [min(max(int(v), 0), T) for v in seq]
    P = len(s) // 2
    et = torch.tensor([float(beta * e[s[i]:s[i + 1]].sum()) for i in range(2 * P)], dtype=torch.float64)
    close(got["reward"], want["reward"], et + 2 * EPS * want["reward"].abs() + 1e-12, "reward")
    h = et[0::2] + et[1::2] + 4 * EPS * (want["reward"].abs()[0::2] + want["reward"].abs()[1::2] + 1)
    close(got["loss"], want["loss"], h + 4 * EPS * (1 + want["loss"]), "loss")
    r = want["result"].double()
    st = torch.stack([(h + 4 * EPS * (1 + torch.nan_to_num(want["loss"]))).sum() / n, h.sum() / n, torch.tensor(0.0).double(),
                      torch.tensor(0.0).double()])
    close(got["result"], r, st + 4 * EPS * r.abs(), "result")
    if backward:
        rel = torch.zeros(T, dtype=torch.float64)
        for p in range(P):
            gp = float(want["g"][s[2 * p]:s[2 * p + 2]].abs().max()) if s[2 * p + 2] > s[2 * p] else 0.0
            if gp > 0 and math.isfinite(gp):
                rel[s[2 * p]:s[2 * p + 2]] = beta * float(h[p]) / 4 / gp + 8 * EPS + min(1.0, float(h[p]))
        w = torch.nan_to_num(want["g"].abs()) * seed / n / tau
        check_dx(got["dx"], want["dx"], dtype, w, rel, hot(y, V), "dx")


@pytest.mark.parametrize("V", [1, 33, 1000, 4097, 32003])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("smooth", [0.0, 0.1])
def test_preference_over_vocabularies(lctx, V, dtype, smooth):
    T = 23
    g, x, y = make(T, V, dtype, 7)
    seq = [1, 5, 9, 9, 12, 20, 22]                # rows outside, an empty sequence, ragged
    y[5:9] = -100 if V == 33 else y[5:9]            # a sequence without valid rows
    ref = (R.logprob(x, y, 1.3) + 0.4 * torch.randn(T, generator=g)).float()
    ref[y < 0] = NAN
    got = run_preference(lctx, x, y, seq, 3, ref, 0.3, smooth, 1.3, 2.0 ** 8, pad=2, lead=1)
    want = R.preference(x, y, seq, 3, ref, 0.3, smooth, 1.3, 2.0 ** 8)
    check_preference(got, want, x, y, seq, 3, dtype, 0.3, 1.3, 2.0 ** 8, ref)


@pytest.mark.parametrize("kw", [dict(in_place=True), dict(in_place=True, pad=7, lead=3), dict(backward=False)])
def test_preference_layouts(lctx, kw):
    T, V = 16, 2500
    g, x, y = make(T, V, "bf16", 8)
    seq = [0, 4, 8, 12, 16]
    got = run_preference(lctx, x, y, seq, 2, None, 0.1, 0.0, 1.0, 1.0, **kw)
    check_preference(got, R.preference(x, y, seq, 2), x, y, seq, 2, "bf16", 0.1, 1.0, 1.0, None, kw.get("backward", True))


def test_preference_large_vocabulary_and_many_pairs(lctx):
    g, x, y = make(4, 128256, "bf16", 9, masked=0.0)
    got = run_preference(lctx, x, y, [0, 1, 2, 3, 4], 2, seed=16.0)
    check_preference(got, R.preference(x, y, [0, 1, 2, 3, 4], 2, seed=16.0), x, y, [0, 1, 2, 3, 4], 2, "bf16", 0.1, 1.0, 16.0, None)
    g, x, y = make(512, 65, "f32", 10)
    seq = list(range(0, 513, 4))
    got = run_preference(lctx, x, y, seq, 64)
    check_preference(got, R.preference(x, y, seq, 64), x, y, seq, 64, "f32", 0.1, 1.0, 1.0, None)


def test_preference_edges(lctx):
    """No pairs, no rows, saturated margins, a NaN row that spoils its own pair alone, and
    offsets outside the rows."""
    g, x, y = make(8, 50, "f32", 11, masked=0.0)
    got = run_preference(lctx, x, y, [0], 1)
    assert got["result"].tolist() == [0.0] * 4 and float(got["dx"].abs().max()) == 0.0
    got = run_preference(lctx, x[:0], y[:0], [0, 0, 0], 1)
    assert abs(float(got["result"][0]) - math.log(2)) < 1e-6 and float(got["result"][3]) == 1
    ref = torch.zeros(8)
    ref[0], ref[2], ref[4], ref[6] = -3e4, 3e4, 3e38, -3e38     # pairs (0,1) won, (2,3) lost by far
    seq = [0, 1, 2, 3, 4]
    got = run_preference(lctx, x, y, seq, 1, ref, 1.0)
    want = R.preference(x, y, seq, 1, ref, 1.0)
    check_preference(got, want, x, y, seq, 1, "f32", 1.0, 1.0, 1.0, ref)
    x[1, 4] = NAN
    got = run_preference(lctx, x, y, [0, 2, 4, 6, 8], 2)
    nan = torch.isnan(got["dx"]).any(1).tolist()
    assert nan == [True] * 4 + [False] * 4 and torch.isnan(got["loss"]).tolist() == [True, False]
    x[1, 4] = 0.0
    got = run_preference(lctx, x, y, [-5, 2, 4, 6, 100], 2)
    want = R.preference(x, y, [0, 2, 4, 6, 8], 2)
    check_preference(got, want, x, y, [0, 2, 4, 6, 8], 2, "f32", 0.1, 1.0, 1.0, None)


# ------------------------------------------------------------------ distillation

def run_distill(lctx, x, teacher, ids, n, y=None, kd=1.0, ce=0.0, tau=1.0, seed=None, pad=0, lead=0, in_place=False,
                backward=True, dpad=None, dlead=None):
    T, V = x.shape
    X = Rows(T, V, x.dtype, pad, lead, x.cuda())
    D = X if in_place else Rows(T, V, x.dtype, pad if dpad is None else dpad, lead if dlead is None else dlead)
    loss, res = torch.full((T,), 77.0, device="cuda"), torch.full((4,), 77.0, device="cuda")
    s = None if seed is None else torch.tensor([seed], device="cuda")
    tl.tl_distill_loss(lctx, X.t, cu(teacher), cu(ids), n, res, targets=cu(y), kd_weight=kd, ce_weight=ce,
                       temperature=tau, seed=s, dlogits=D.t if backward else None, row_loss=loss)
    torch.cuda.synchronize()
    assert X.outside_untouched() and D.outside_untouched()
    return {"loss": loss, "result": res, "dx": D.t}


def check_distill(got, want, x, teacher, ids, y, n, dtype, kd, ce, tau, seed, backward=True):
    T, V = x.shape
    big = 1.0
    for m in (x, teacher):
        if m is not None and m.numel():
            f = m.double()[torch.isfinite(m.double()) & (m.double().abs() < 1e30)]
            big = max(big, float(f.abs().max()) / tau if f.numel() else 1.0)
    valid = torch.ones(T, dtype=torch.bool) if y is None else y >= 0
    tol = kd * tau ** 2 * (2 * REL + 16 * EPS * big) + ce * (2 * REL + 16 * EPS * big * tau) + 4 * EPS * torch.nan_to_num(want["loss"].abs())
    tol = torch.where(valid, tol, 0.0)
    close(got["loss"], want["loss"], tol, "loss")
    want_r = want["result"].double()
    each = 2 * REL + 16 * EPS * big * max(1.0, tau)
    st = torch.tensor([float(tol.sum()) / n, tau ** 2 * each * T / n, each * T / n, 0.0], dtype=torch.float64)
    close(got["result"], want_r, st + 4 * EPS * torch.nan_to_num(want_r.abs()), "result")
    if backward:
        listed = torch.zeros(T, V, dtype=torch.bool) if y is None else hot(y, V)
        if ids is not None:
            for t in range(T):
                for j in ids[t].tolist():
                    if 0 <= j < V:
                        listed[t, j] = True
        w = torch.full((T,), seed / n * (kd * tau + ce), dtype=torch.float64) * valid
        check_dx(got["dx"], want["dx"], dtype, w, torch.full((T,), 2 * REL + 64 * EPS, dtype=torch.float64) * valid, listed, "dx")


def teacher_of(T, V, K, g, dtype="f32", wide=False):
    ids = torch.stack([torch.randperm(V, generator=g)[:K] for _ in range(T)]) if K <= V else \
        torch.randint(0, V, (T, K), generator=g)
    t = (torch.randn(T, K, generator=g) * 3).to(DT[dtype])
    return t, (ids if wide else ids.int())


@pytest.mark.parametrize("V", [1, 2, 33, 1000, 4097, 32003])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("tau,kd,ce,K", [(1.0, 1.0, 0.0, 8), (2.0, 0.7, 0.3, 17), (0.7, 1.0, 1.0, 1), (1.0, 0.5, 0.5, 33),
                                         (3.0, 0.6, 0.4, 5), (4.0, 0.6, 0.4, 300)])
def test_distill_over_vocabularies(lctx, V, dtype, tau, kd, ce, K):
    T = 7
    g, x, y = make(T, V, dtype, 12)
    teacher, ids = teacher_of(T, V, min(K, V), g, dtype, wide=K % 2 == 1)
    got = run_distill(lctx, x, teacher, ids, 5, y, kd, ce, tau, 2.0 ** 6, pad=1, lead=1)
    want = R.distill(x, teacher, ids, 5, y, kd, ce, tau, 2.0 ** 6)
    check_distill(got, want, x, teacher, ids, y, 5, dtype, kd, ce, tau, 2.0 ** 6)


@pytest.mark.parametrize("V,dtype", [(128256, "bf16"), (128256, "f32"), (300001, "f16")])
def test_distill_large_vocabulary(lctx, V, dtype):
    g, x, y = make(3, V, dtype, 13, masked=0.0)
    teacher, ids = teacher_of(3, V, 64, g, "bf16")
    for in_place in (False, True):
        got = run_distill(lctx, x, teacher, ids, 3, y, 0.75, 0.25, 2.0, 1.0, in_place=in_place)
        check_distill(got, R.distill(x, teacher, ids, 3, y, 0.75, 0.25, 2.0), x, teacher, ids, y, 3, dtype, 0.75, 0.25, 2.0, 1.0)


def test_distill_teacher_edges(lctx):
    """Padded ids, equal ids (within the list and with the label), rows without entries,
    teacher logits of -inf, ids beyond the vocabulary, excluded student tokens, NaN in what
    is not read."""
    T, V, K = 9, 700, 6
    g, x, y = make(T, V, "f32", 14, masked=0.0)
    teacher, ids = teacher_of(T, V, K, g)
    ids[0] = torch.tensor([3, 3, 3, 5, 5, 9]); y[0] = 5
    ids[1, 2:] = -1; teacher[1, 2:] = NAN                # padding, whatever its logits
    ids[2] = -1                                        # no entries
    teacher[3] = -INF                                  # nothing left of the teacher
    teacher[4, :5] = -INF                              # one entry left
    x[4, ids[4, 0].item()] = -INF                      # excluded by both
    x[5, ids[5, 1].item()] = -INF                      # excluded by the student alone: kd = inf
    ids[6, 3] = V                                      # not an id
    ids[7, 3], teacher[7, 3] = y[7].int(), 9.0           # the label listed
    y[8] = -3; x[8] = NAN; teacher[8] = NAN; ids[8] = V + 5
    for in_place in (False, True):
        for kd, ce in ((1.0, 0.0), (0.6, 0.4)):
            got = run_distill(lctx, x, teacher, ids, 8, y, kd, ce, 2.0, 4.0, in_place=in_place)
            want = R.distill(x, teacher, ids, 8, y, kd, ce, 2.0, 4.0)
            assert float(want["loss"][5]) == INF and math.isnan(float(want["loss"][6]))
            check_distill(got, want, x, teacher, ids, y, 8, "f32", kd, ce, 2.0, 4.0)


def test_distill_without_targets_and_cross_entropy_alone(lctx):
    g, x, y = make(6, 999, "bf16", 15)
    teacher, ids = teacher_of(6, 999, 1000 % 64, g)
    got = run_distill(lctx, x, teacher, ids, 6, None, 1.0, 0.0, 1.5, 2.0)
    check_distill(got, R.distill(x, teacher, ids, 6, None, 1.0, 0.0, 1.5, 2.0), x, teacher, ids, None, 6, "bf16", 1.0, 0.0, 1.5, 2.0)
    got = run_distill(lctx, x, None, None, 4, y, 1.0, 1.0, 1.0, 2.0, dpad=3, dlead=1)
    check_distill(got, R.distill(x, None, None, 4, y, 1.0, 1.0, 1.0, 2.0), x, None, None, y, 4, "bf16", 1.0, 1.0, 1.0, 2.0)
    got = run_distill(lctx, x, teacher, ids, 4, y, 0.0, 1.0, 1.0, 2.0, backward=False)
    check_distill(got, R.distill(x, teacher, ids, 4, y, 0.0, 1.0, 1.0, 2.0), x, teacher, ids, y, 4, "bf16", 0.0, 1.0, 1.0, 2.0, False)


def test_distill_most_entries_in_few_rows(lctx):
    g, x, y = make(2, 5000, "f16", 16, masked=0.0)
    teacher, ids = teacher_of(2, 5000, 1024, g)
    ids[1] = ids[1] % 300                              # many equal ids
    got = run_distill(lctx, x, teacher, ids, 2, y, 0.5, 0.5, 1.0, 2.0 ** 12)
    check_distill(got, R.distill(x, teacher, ids, 2, y, 0.5, 0.5, 1.0, 2.0 ** 12), x, teacher, ids, y, 2, "f16", 0.5, 0.5, 1.0, 2.0 ** 12)


# ------------------------------------------------------------------ what all share

@pytest.mark.parametrize("op", ["policy", "preference", "distill"])
def test_gradient_against_differences_of_the_loss(lctx, op):
    """The directional derivative of the kernel's own forward.  With a step h along d the
    difference carries 2 tol(loss) / 2h of rounding and h^2 / 6 of a third derivative whose
    magnitude along a unit-size d stays below 1: at h = 0.05, 2.5e-5 / 0.05 + 4e-4 = 9e-4."""
    T, V, h = 8, 300, 0.05
    g, x, y = make(T, V, "f32", 17, masked=0.2)
    d = torch.randn(T, V, generator=g)
    d = d / d.norm()
    lp = R.logprob(x, y)
    old, adv = (lp - 0.05).float(), torch.linspace(0.5, 1.5, T)
    teacher, ids = teacher_of(T, V, 9, g)

    def call(v, back):
        if op == "policy":
            return run_policy(lctx, v, y, old, adv, 4, backward=back)
        if op == "preference":
            return run_preference(lctx, v, y, [0, 2, 4, 6, 8], 2, beta=0.5, backward=back)
        return run_distill(lctx, v, teacher, ids, 4, y, 0.7, 0.3, 2.0, backward=back)

    slope = float((call(x, True)["dx"].double().cpu() * d.double()).sum())
    up, down = (float(call(x + s * h * d, False)["result"][0].double()) for s in (1, -1))
    assert abs((up - down) / (2 * h) - slope) < 9e-4


def test_results_repeat_bit_for_bit_and_in_a_graph_and_on_another_stream(lctx):
    T, V = 300, 5003
    g, x, y = make(T, V, "bf16", 18)
    X, Y = x.cuda(), y.cuda()
    lp = R.logprob(x, y)
    old, adv = (lp + 0.2 * torch.randn(T, generator=g)).float().cuda(), torch.randn(T, generator=g).cuda()
    teacher, ids = (t.cuda() for t in teacher_of(T, V, 20, g))
    seq = torch.arange(0, T + 1, 10, device="cuda")
    seed = torch.tensor([2.0], device="cuda")
    outs = [torch.zeros_like(X) for _ in range(3)]
    res = [torch.zeros(4, device="cuda") for _ in range(3)]

    def calls(stream=None):
        tl.tl_policy_loss(lctx, X, Y, old, adv, 200, res[0], seed=seed, dlogits=outs[0], stream=stream)
        tl.tl_preference_loss(lctx, X, Y, seq, 15, res[1], seed=seed, dlogits=outs[1], stream=stream)
        tl.tl_distill_loss(lctx, X, teacher, ids, 200, res[2], targets=Y, ce_weight=0.5, temperature=2.0, seed=seed,
                           dlogits=outs[2], stream=stream)

    calls()
    first = [t.clone() for t in outs + res]
    for t in outs + res:
        t.zero_()
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    calls(other)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, outs + res))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    for t in outs + res:
        t.zero_()
    seed.fill_(4.0)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    # a seed twice as large doubles every gradient exactly (bf16 normals), the losses stay
    assert all(torch.equal(a, b) for a, b in zip(first[3:], res))
    assert all(torch.equal(2 * a, b) for a, b in zip(first[:3], outs))


@pytest.mark.parametrize("V", [1, 7, 33, 257, 1000, 1025, 2040, 4096, 4290])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_many_rows(lctx, V, dtype):
    """Over a thousand rows, where the short ones take a warp each: every operator that has
    that form, at every row phase, masks and non-finite rows among them, in place and not."""
    T = 1061
    g, x, y = make(T, V, dtype, 21)
    low = torch.finfo(DT[dtype]).min
    x[3], y[3] = -INF, 0
    x[4], y[4] = low, 0
    x[5, V - 1], y[5] = NAN, 0
    y[6] = V
    x[7, 0], y[7] = INF, 0
    x[8], y[8] = NAN, -1
    good = torch.ones(T, dtype=torch.bool)
    good[torch.tensor([3, 5, 6, 7])] = False
    lp = R.logprob(x, y)
    old = (torch.nan_to_num(lp, nan=0.0) + 0.2 * torch.randn(T, generator=g)).float()
    adv, ref = torch.randn(T, generator=g), (torch.nan_to_num(lp, nan=0.0) + 0.3).float()
    for kw in (dict(pad=3, lead=1), dict(in_place=True)):
        got = run_policy(lctx, x, y, old, adv, 900, ref, 0.05, seed=64.0, **kw)
        want = R.policy(x, y, old, adv, 900, ref, kl_weight=0.05, seed=64.0)
        check_policy(got, want, x, y, old, adv, 900, dtype, 1.0, 64.0, 0.05, ref)
    X, out = Rows(T, V, DT[dtype], 5, 2, x.cuda()), torch.full((T,), 9.0, device="cuda")
    tl.tl_token_logprob(lctx, X.t, y.cuda(), out)
    close(out, lp, lp_tol(lp), "logp")
    # preference: the bad rows in a pair of their own
    seq = [0, 4, 9, 100, 200, 500, 1061]
    got = run_preference(lctx, x, y, seq, 3, ref, 0.02, 0.0, 1.0, 32.0, pad=1)
    want = R.preference(x, y, seq, 3, ref, 0.02, 0.0, 1.0, 32.0)
    check_preference(got, want, x, y, seq, 3, dtype, 0.02, 1.0, 32.0, ref)


def test_offsets_beyond_32_bits(lctx):
    """Rows 2^29 elements apart: the last starts at element 2^32."""
    T, V, ld = 9, 1000, 1 << 29
    buf = torch.empty((T - 1) * ld + V, dtype=torch.bfloat16, device="cuda")
    X = torch.as_strided(buf, (T, V), (ld, 1))
    g, x, y = make(T, V, "bf16", 19, masked=0.0)
    X.copy_(x.cuda())
    lp = R.logprob(x, y)
    old, adv = (lp + 0.1).float(), -torch.ones(T)
    res, got_lp = torch.zeros(4, device="cuda"), torch.zeros(T, device="cuda")
    tl.tl_policy_loss(lctx, X, y.cuda(), old.cuda(), adv.cuda(), T, res, dlogits=X, logp=got_lp)
    loss = torch.zeros(T, device="cuda")
    want = R.policy(x, y, old, adv, T)
    close(got_lp, want["logp"], lp_tol(want["logp"]), "logp")
    w = want["g"].abs() / T
    check_dx(X, want["dx"], "bf16", w, torch.full((T,), 1e-4, dtype=torch.float64), hot(y, V), "dx")
    del loss, buf


def test_refusals_launch_nothing(lctx):
    T, V = 4, 64
    x = torch.zeros(T, V, device="cuda")
    y = torch.zeros(T, dtype=torch.int64, device="cuda")
    f, res, d = torch.zeros(T, device="cuda"), torch.zeros(4, device="cuda"), torch.zeros(T, V, device="cuda")
    ids, tea = torch.zeros(T, 2, dtype=torch.int32, device="cuda"), torch.zeros(T, 2, device="cuda")
    g, old = torch.zeros(T, device="cuda"), torch.zeros(T, device="cuda")
    before = tl.tl_loss_launch_count(lctx)
    pol = lambda **k: tl.tl_policy_loss(lctx, k.pop("x", x), k.pop("y", y), old, g, k.pop("n", 4), k.pop("res", res), **k)  # noqa: E731
    dis = lambda **k: tl.tl_distill_loss(lctx, x, k.pop("tea", tea), k.pop("ids", ids), 4, res, **k)  # noqa: E731
    pre = lambda **k: tl.tl_preference_loss(lctx, x, y, k.pop("seq", torch.tensor([0, 2, 4], device="cuda")), 1, res, **k)  # noqa: E731
    for call in (lambda: pol(n=0), lambda: pol(temperature=0.0), lambda: pol(temperature=-1.0), lambda: pol(temperature=NAN),
                 lambda: pol(temperature=INF), lambda: pol(clip_low=1.5), lambda: pol(clip_high=-0.1), lambda: pol(clip_high=NAN),
                 lambda: pol(kl_weight=-1.0, ref_logp=f), lambda: pol(kl_weight=0.1), lambda: pol(logp=old), lambda: pol(logp=f, row_loss=f),
                 lambda: pol(dlogits=x, logp=x[0, :T]), lambda: pol(dlogits=d, seed=d[0, :1]),
                 lambda: pol(x=x[:, :32], dlogits=x[:, 16:48]),
                 lambda: pol(x=x.expand(T, V)[:1].expand(T, V)),
                 lambda: pre(beta=0.0), lambda: pre(beta=-1.0), lambda: pre(label_smoothing=0.6), lambda: pre(label_smoothing=NAN),
                 lambda: dis(ce_weight=0.5), lambda: dis(kd_weight=-1.0), lambda: dis(ids=torch.zeros(T, 2, dtype=torch.int16, device="cuda")),
                 lambda: dis(tea=torch.zeros(T, 1025, device="cuda"), ids=torch.zeros(T, 1025, dtype=torch.int32, device="cuda")),
                 lambda: dis(tea=tea.double())):
        with pytest.raises(tl.TLError) as e:
            call()
        assert e.value.status == tl.TL_EINVAL and len(str(e.value)) > 30
    for call in (lambda: pol(y=y.int()), lambda: pol(y=y[:3]), lambda: pol(res=res[:3]), lambda: pol(x=x.double()),
                 lambda: pol(x=x.t()), lambda: pol(x=x[0]), lambda: pol(dlogits=d.half()), lambda: pol(dlogits=d[:3]),
                 lambda: pol(y=y.cpu()), lambda: pre(seq=torch.zeros(4, dtype=torch.int64, device="cuda")),
                 lambda: dis(ids=ids[:3]), lambda: dis(tea=torch.zeros(T, 3, device="cuda"))):
        with pytest.raises(ValueError):
            call()
    small = tl.tl_loss_create(2)
    with pytest.raises(tl.TLError):
        tl.tl_token_logprob(small, x, y, f)                       # more rows than the context holds
    with pytest.raises(tl.TLError):
        tl.tl_preference_loss(small, x[:2], y[:2], torch.tensor([0, 1, 2], device="cuda"), 1, res)
    tl.tl_loss_destroy(small)
    with pytest.raises(tl.TLError):
        tl.tl_token_logprob(small, x[:1], y[:1], f[:1])
    assert tl.tl_loss_launch_count(lctx) == before
    # columns of one matrix may hold logits and gradient side by side
    both = torch.randn(T, 2 * V, device="cuda")
    tl.tl_policy_loss(lctx, both[:, :V], y, old, g, 4, res, dlogits=both[:, V:])
    torch.cuda.synchronize()


def test_example_trains_with_every_objective(lctx):
    """The example end to end: the objectives' gradients, scaled on the device, through the
    optimizer step.  Each loss falls and no update is lost to an overflow that sticks."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "post_training.py")
    spec = importlib.util.spec_from_file_location("post_training", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    for name in ("distill", "preference", "policy"):
        losses, status = example.train(name, 30, lctx)
        assert all(math.isfinite(v) for v in losses), name
        assert losses[-1] < losses[0], name
        assert status.t >= 25 and status.found_inf == 0, name
