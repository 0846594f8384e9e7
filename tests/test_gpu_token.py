"""Row statistics and their gradient on the GPU against their fp64 statements (token_reference.py).

Tolerances (eps = 2^-24; REL = 2.5e-5 bounds the relative error of a row's sum S, of q where it carries the sum and
the absolute error of log S: the exponent of a term, at most 30 bits where it matters, rounds three times, 0.69 * 90
eps = 3.7e-6, the exponential adds 2^-22, and sums run in chains of at most 256 terms, 1.5e-5):
* log q of an element: REL + 4 eps |log q|.
* entropy = log S + D with D = sum q (max - x) / tau: log S as above, D the quotient of two sums of terms with the
  same errors: REL + 2 REL D + 8 eps (log S + D).
* gradient step q (a + b (log q + H)): q within 2 REL, the bracket within |b| (errors of log q and H) plus 4 eps of its
  parts; + step a at the label, 4 eps; rounded once to the type.  Exponentials below 2^-126 are 0.
Ids are whole numbers and have to be equal.
"""
import pytest

torch = pytest.importorskip("torch")

import loss_scaled_adamw_gb300 as tl
import token_reference as R

pytestmark = pytest.mark.gpu

EPS, REL = 2.0 ** -24, 2.5e-5
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lctx():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from loss_scaled_adamw_gb300 import _build
    _build.build()
    return tl.tl_loss_create(20000)


def place(x, pad=0, lead=0):
    """A device copy of x whose rows are `pad` elements apart and start `lead` elements into a buffer."""
    T, V = x.shape
    buf = torch.full((lead + T * (V + pad) + 8,), 12345.0, dtype=x.dtype, device="cuda")
    t = buf[lead:lead + T * (V + pad)].view(T, V + pad)[:, :V]
    t.copy_(x)
    return t, buf


def run(lctx, x, y, k, tau=1.0, wide=False, pad=0, lead=0, gap=0, stream=None):
    T = x.shape[0]
    xd, _ = place(x, pad, lead)
    f = lambda *s: torch.full(s, 7.0, device="cuda")  # noqa: E731
    ids = torch.full((T, k + gap), 77, dtype=torch.int64 if wide else torch.int32, device="cuda")
    top = f(T, k + gap)
    out = {"logp": f(T) if y is not None else None, "entropy": f(T), "saved": f(T, 3)}
    kw = dict(top_ids=ids[:, :k], top_logp=top[:, :k]) if k else {}
    tl.tl_token_stats(lctx, xd, targets=None if y is None else y.cuda(), temperature=tau, stream=stream, **out, **kw)
    torch.cuda.synchronize()
    assert (ids[:, k:] == 77).all() and (top[:, k:] == 7.0).all()
    out.update(ids=ids[:, :k].cpu().long(), top=top[:, :k].cpu())
    return xd, {n: v.cpu() for n, v in out.items() if v is not None}


def close(got, want, tol, what):
    got, want = got.double(), want.double()
    assert torch.equal(torch.isnan(got), torch.isnan(want)), what
    inf = torch.isinf(want)
    assert torch.equal(got[inf], want[inf]), what
    off = (got - want).abs()
    bad = ~(off <= tol) & ~torch.isnan(want) & ~inf
    assert not bad.any(), (what, got[bad][:4], want[bad][:4], off[bad].max())


def entropy_tol(want):
    gap = want["entropy"] - want["saved"][:, 1]      # D
    return REL + 2 * REL * gap.abs() + 8 * EPS * (want["saved"][:, 1].abs() + gap.abs())


def compare(got, want):
    assert torch.equal(got["ids"], want["ids"]), (got["ids"], want["ids"])
    log_tol = lambda v: REL + 4 * EPS * v.abs()  # noqa: E731
    if "logp" in got:
        close(got["logp"], want["logp"], log_tol(want["logp"]), "logp")
    close(got["top"], want["top"], log_tol(want["top"]), "top")
    close(got["entropy"], want["entropy"], entropy_tol(want), "entropy")
    close(got["saved"][:, 0], want["saved"][:, 0], 0.0, "max")
    close(got["saved"][:, 1], want["saved"][:, 1], log_tol(want["saved"][:, 1]), "log_sum")
    assert torch.equal(torch.nan_to_num(got["saved"][:, 2], 1e9), torch.nan_to_num(got["entropy"], 1e9))


def make(T, V, dtype, seed, masked=0.25, spread=3.0):
    g = torch.Generator().manual_seed(1000 * seed + 7 * T + V)
    x = torch.randn(T, V, generator=g) * spread
    y = torch.randint(0, V, (T,), generator=g)
    for t in range(T):
        x[t, y[t]] += 4.0
    if T > 1:
        y = torch.where(torch.rand(T, generator=g) < masked, -100, y)
    return x.to(DT[dtype]), y


SHAPES = [(1, 1), (3, 2), (5, 7), (4, 16), (7, 33), (9, 255), (20, 1000), (3, 2049), (6, 4099), (5, 8192), (3, 12345),
          (3, 40000), (2, 80003), (2, 128256), (1, 300001)]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T,V", SHAPES)
def test_shapes(lctx, T, V, dtype):
    for i, k in enumerate((0, 1, 5, 64, 256)):
        x, y = make(T, V, dtype, i)
        tau = (1.0, 0.7, 2.0)[i % 3]
        _, got = run(lctx, x, y, k, tau, wide=i % 2 == 1, pad=(0, 3, 8)[i % 3], lead=(0, 1, 5)[i % 3], gap=i % 3)
        compare(got, R.stats(x, y, k, tau))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V,rows", [(500, 300), (1000, 700), (1003, 260), (2001, 600), (4096, 520), (5001, 900), (9000, 400)])
def test_many_rows(lctx, V, rows, dtype):
    """Enough rows for every form of the kernel: twenty rows, again and again."""
    base, y0 = make(20, V, dtype, 3)
    x, y = base.repeat(rows // 20, 1), y0.repeat(rows // 20)
    for k in (0, 3, 40, 256):
        _, got = run(lctx, x, y, k, 1.0)
        want = R.stats(base, y0, k)
        compare(got, {n: v.repeat(rows // 20, *[1] * (v.dim() - 1)) for n, v in want.items()})


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("V,rows", [(17000, 700), (33001, 640), (50001, 400), (128256, 200)])
def test_many_long_rows(lctx, V, rows, dtype):
    """Rows whose entries some warps choose while others read the next ones; among them rows whose choice takes far
    longer than the others' (equal entries, the largest side by side), ignored ones and ones without a softmax."""
    base, y0 = make(10, V, dtype, 3, masked=0.0)
    base[2] = 0.5
    base[5] = torch.linspace(-4, 4, V).to(base.dtype)
    base[7, 11] = NAN
    base[8] = torch.randint(0, 3, (V,), generator=torch.Generator().manual_seed(1)).to(base.dtype)
    y0[3] = y0[4] = -1
    order = torch.randint(0, 10, (rows,), generator=torch.Generator().manual_seed(V))
    order[:10] = torch.arange(10)
    for k in (1, 40, 256):
        _, got = run(lctx, base[order], y0[order], k, wide=k == 40)
        compare(got, {n: v[order] for n, v in R.stats(base, y0, k).items()})


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("V", [40, 1001, 5000, 40003, 128256])
@pytest.mark.parametrize("times", [1, 50])
def test_masks_and_rows_without_a_softmax(lctx, V, dtype, times):
    times = min(times, max(1, 2000000 // V))
    x, _ = make(12, V, dtype, 5)
    low = torch.finfo(DT[dtype]).min
    x[0] = -INF                                     # nothing but excluded tokens
    x[1] = -INF
    x[1, V // 3] = 1.5                              # one token
    x[2] = -INF
    x[2, V - 7:] = torch.arange(7).to(x.dtype)      # seven at the end
    x[3, 5] = NAN
    x[4, V - 1] = INF
    x[5] = low                                      # nothing but the lowest value: a uniform row
    x[6] = low
    x[6, 3], x[6, V - 2] = 2.0, 1.0
    x[7, : V // 2] = low
    x[8, ::2] = -INF
    x[9] = -3.0e4                                   # a mask value in every type
    x[9, V // 2] = 0.25
    x[10, :] = NAN
    y = torch.tensor([1, V // 3, 0, 1, 2, 3, V - 2, 4, 1, V // 2, 0, V + 5])
    for k in (0, 6, 30):
        _, got = run(lctx, x.repeat(times, 1), y.repeat(times), k)
        want = R.stats(x, y, k)
        compare(got, {n: v.repeat(times, *[1] * (v.dim() - 1)) for n, v in want.items()})


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("V,times", [(37, 1), (37, 70), (1000, 1), (1000, 70), (4100, 1), (4100, 70), (30011, 1), (128256, 1)])
def test_ties_and_orders(lctx, V, times, dtype):
    g = torch.Generator().manual_seed(V)
    x = torch.zeros(8, V, dtype=DT[dtype])
    x[0] = 0.75                                                            # all equal
    x[1] = torch.randint(0, 3, (V,), generator=g).to(x.dtype)              # three values
    x[2] = (torch.arange(V) * 8 // V).to(x.dtype)                          # ascending steps
    x[3] = -(torch.arange(V) * 8 // V).to(x.dtype)                         # descending
    x[4] = torch.linspace(-4, 4, V).to(x.dtype)                            # ascending, the largest side by side
    x[5] = torch.where(torch.arange(V) % 2 == 0, 0.0, -0.0).to(x.dtype)    # zeros of both signs are equal
    x[6] = -torch.rand(V, generator=g).to(x.dtype)
    x[6, V // 2:] = x[6, : V - V // 2].clone()                             # every value twice
    x[7, : min(V, 300)] = torch.arange(min(V, 300)).to(x.dtype) / 64       # the first 300 hold the largest
    y = torch.arange(8) % V
    for k in (1, 20, 100, 256):
        _, got = run(lctx, x.repeat(times, 1), y.repeat(times), k)
        want = R.stats(x, y, k)
        compare(got, {n: v.repeat(times, *[1] * (v.dim() - 1)) for n, v in want.items()})


@pytest.mark.parametrize("dtype,offset", [("f32", 1e4), ("f32", -3e6), ("f32", 1e12), ("bf16", -2.0 ** 13), ("f16", 6e4), ("f32", -1e9)])
@pytest.mark.parametrize("V", [901, 3001, 20000])
def test_offsets(lctx, dtype, offset, V):
    g = torch.Generator().manual_seed(9)
    x = (torch.randn(4, V, generator=g) * 4 + offset).to(DT[dtype])
    y = torch.tensor([0, 7, -1, V - 1])
    for tau in (1.0, 2.0):
        for times in (1, 130):
            _, got = run(lctx, x.repeat(times, 1), y.repeat(times), 9, tau)
            want = R.stats(x, y, 9, tau)
            compare(got, {n: v.repeat(times, *[1] * (v.dim() - 1)) for n, v in want.items()})


def test_without_targets_and_single_outputs(lctx):
    x, _ = make(6, 777, "bf16", 1)
    _, got = run(lctx, x, None, 4)
    compare(got, R.stats(x, None, 4))
    xd, y = x.cuda(), torch.tensor([3, 5, -1, 700, 0, 776]).cuda()
    want, free = R.stats(x, y.cpu(), 2), R.stats(x, None)
    e = torch.full((6,), 7.0, device="cuda")
    tl.tl_token_stats(lctx, xd, entropy=e)
    close(e.cpu(), free["entropy"], entropy_tol(free), "entropy alone")
    lp = torch.full((6,), 7.0, device="cuda")
    tl.tl_token_stats(lctx, xd, targets=y, logp=lp)
    close(lp.cpu(), want["logp"], REL + 4 * EPS * want["logp"].abs(), "logp alone")
    ids, top = torch.zeros(6, 2, dtype=torch.int32, device="cuda"), torch.zeros(6, 2, device="cuda")
    tl.tl_token_stats(lctx, xd, targets=y, top_ids=ids, top_logp=top)
    assert torch.equal(ids.cpu().long(), want["ids"])


def test_refusals(lctx):
    x = torch.zeros(4, 50, device="cuda")
    y = torch.zeros(4, dtype=torch.int64, device="cuda")
    f = lambda *s: torch.zeros(*s, device="cuda")  # noqa: E731
    i = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    before = tl.tl_loss_launch_count(lctx)
    for kw in (dict(), dict(logp=f(4)), dict(top_ids=i(4, 257), top_logp=f(4, 257)), dict(entropy=x[0, :4]),
               dict(top_ids=x.view(torch.int32)[:, :2], top_logp=x[:, 2:4])):
        with pytest.raises(tl.TLError):
            tl.tl_token_stats(lctx, x, **kw)
    shared = f(12)
    with pytest.raises(tl.TLError):
        tl.tl_token_stats(lctx, x, targets=y, logp=shared[:4], saved=shared.view(4, 3))
    for kw in (dict(top_ids=i(4, 2)), dict(top_logp=f(4, 2)), dict(top_ids=i(4, 2), top_logp=f(4, 3)),
               dict(top_ids=i(4, 2), top_logp=f(4, 2).double()), dict(saved=f(12)), dict(saved=f(3, 4)), dict(entropy=f(5)),
               dict(entropy=f(4).cpu()), dict(targets=y.int(), logp=f(4))):
        with pytest.raises(ValueError):
            tl.tl_token_stats(lctx, x, **kw)
    with pytest.raises(tl.TLError):
        tl.tl_token_stats(lctx, x, top_ids=i(4, 2).short(), top_logp=f(4, 2))
    d, s = torch.zeros_like(x), f(4, 3)
    for kw in (dict(), dict(grad_logp=f(4)), dict(targets=y, grad_logp=f(4), temperature=0.0)):
        with pytest.raises(tl.TLError):
            tl.tl_token_grad(lctx, x, s, d, **kw)
    with pytest.raises(tl.TLError):
        tl.tl_token_grad(lctx, x, None, d, grad_entropy=f(4))
    with pytest.raises(tl.TLError):
        tl.tl_token_grad(lctx, x, s, None, grad_entropy=f(4))
    with pytest.raises(tl.TLError):      # shifted against the logits
        flat = f(250)
        tl.tl_token_grad(lctx, flat[:200].view(4, 50), s, flat[50:].view(4, 50), grad_entropy=f(4))
    with pytest.raises(ValueError):
        tl.tl_token_grad(lctx, x, s, d.half(), grad_entropy=f(4))
    with pytest.raises(ValueError):
        tl.tl_token_grad(lctx, x, s, d, grad_entropy=f(4), seed=0)
    assert tl.tl_loss_launch_count(lctx) == before
    tl.tl_token_stats(lctx, x[:0], entropy=f(0))
    assert tl.tl_loss_launch_count(lctx) == before


# ------------------------------------------------------------------ the gradient

def check_grad(lctx, x, y, ga, gb, tau=1.0, seed=None, pad=0, lead=0, in_place=False, dpad=None):
    T, V = x.shape
    xd, _ = place(x, pad, lead)
    yd = None if y is None else y.cuda()
    saved = torch.zeros(T, 3, device="cuda")
    tl.tl_token_stats(lctx, xd, targets=yd, saved=saved, temperature=tau)
    d, buf = place(torch.zeros_like(x), pad if dpad is None else dpad, lead)
    if in_place:
        d = xd
    else:
        d.fill_(55.0)
    s = None if seed is None else torch.tensor([seed], device="cuda")
    dev = lambda v: None if v is None else v.float().cuda()  # noqa: E731
    tl.tl_token_grad(lctx, xd, saved, d, targets=yd, grad_logp=dev(ga), grad_entropy=dev(gb), temperature=tau, seed=s)
    torch.cuda.synchronize()
    S = 1.0 if seed is None else seed
    want, st = R.grad(x, y, ga, gb, tau, S), R.stats(x, y, 0, tau)
    a, b = (torch.zeros(T, dtype=torch.float64) if v is None else v.double() for v in (ga, gb))
    log_q = (x.double() - st["saved"][:, :1]) / tau - st["saved"][:, 1:2]
    log_q = torch.where(log_q > -INF, log_q, 0.0)
    q = torch.exp(torch.where(x > -INF, log_q, -INF))
    htol = entropy_tol(st)[:, None] + REL + 4 * EPS * log_q.abs()
    bracket = a[:, None].abs() + b[:, None].abs() * (log_q.abs() + st["entropy"][:, None].abs())
    step = abs(S) / tau
    tol = step * q * (2 * REL * bracket + b[:, None].abs() * htol) + step * a[:, None].abs() * 4 * EPS * (q > 1e-30)
    tol = tol + step * bracket * 2.0 ** -126 * 4 + want.abs() * torch.finfo(x.dtype).eps / 2 * 1.01
    tol = tol + {torch.float16: 2.0 ** -25, torch.bfloat16: 1e-38, torch.float32: 1e-38}[x.dtype]
    if y is not None:
        tol[torch.arange(T), y.clamp(0, V - 1)] += step * a.abs() * 4 * EPS
    close(d.cpu(), want, torch.nan_to_num(tol, 0.0), "dlogits")
    if not in_place:
        used = torch.zeros_like(buf, dtype=torch.bool)
        p = pad if dpad is None else dpad
        used[lead:lead + T * (V + p)].view(T, V + p)[:, :V] = True
        assert (buf[~used] == 12345.0).all()
    return d


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T,V", [(1, 1), (3, 2), (5, 7), (7, 33), (9, 255), (20, 1000), (3, 4099), (5, 8192), (3, 40000), (2, 128256)])
def test_gradient(lctx, T, V, dtype):
    g = torch.Generator().manual_seed(V)
    for i, which in enumerate(((True, True), (True, False), (False, True))):
        x, y = make(T, V, dtype, 10 + i)
        ga = torch.randn(T, generator=g) if which[0] else None
        gb = torch.randn(T, generator=g) if which[1] else None
        check_grad(lctx, x, y if which[0] or i else None, ga, gb, (1.0, 0.7, 2.0)[i], (None, 64.0, 3.0)[i], (0, 3, 8)[i],
                   (0, 1, 5)[i], in_place=i == 0, dpad=(0, 4, 8)[i])


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_gradient_of_masked_rows(lctx, dtype):
    V = 1003
    x, _ = make(9, V, dtype, 2)
    x[0] = -INF
    x[1, 3:] = -INF
    x[2, 9] = NAN
    x[3, 9] = INF
    x[4] = torch.finfo(DT[dtype]).min
    x[5, ::2] = torch.finfo(DT[dtype]).min
    x[6] = -INF
    x[6, 44] = 2.0                                  # one token: no gradient anywhere
    y = torch.tensor([0, 2, 1, 1, 5, 1, 44, V, -5])
    g = torch.Generator().manual_seed(1)
    check_grad(lctx, x, y, torch.randn(9, generator=g), torch.randn(9, generator=g))
    zero = torch.zeros(9)
    d = check_grad(lctx, x, y, zero, zero)
    nan = torch.isnan(d).all(1).tolist()
    assert nan == [True, False, True, True, False, False, False, True, False]
    assert (d[[1, 4, 5, 6, 8]] == 0).all()


def test_gradient_against_differences(lctx):
    """The forward's own entropies and log-probabilities, fp32, a step of 2^-5: central differences are off by
    h^2 / 6 times the third derivative (at most 2 here) and by two roundings of the values over 2 h."""
    x, y = make(3, 9, "f32", 4, masked=0.0)
    g = torch.Generator().manual_seed(2)
    ga, gb = torch.randn(3, generator=g), torch.randn(3, generator=g)
    d = check_grad(lctx, x, y, ga, gb).cpu().double()
    h = 2.0 ** -5
    for t in range(3):
        for j in range(9):
            value = []
            for sign in (1, -1):
                z = x.clone()
                z[t, j] += sign * h
                _, got = run(lctx, z, y, 0)
                value.append(float((ga.double() * got["logp"].double() + gb.double() * got["entropy"].double()).sum()))
            weight = float(ga[t].abs() + gb[t].abs())
            assert abs((value[0] - value[1]) / (2 * h) - float(d[t, j])) < weight * (h * h * 2 + 2 * REL / h)


# ------------------------------------------------------------------ streams, graphs, repetition

@pytest.mark.parametrize("T,V", [(700, 5003), (900, 1000), (400, 33001), (3, 60000)])
def test_repeats_bit_for_bit_on_other_streams(lctx, T, V):
    x, y = make(T, V, "bf16", 8)
    _, first = run(lctx, x, y, 33)
    side = torch.cuda.Stream()
    for stream in (side, torch.cuda.current_stream(), side):
        with torch.cuda.stream(stream):
            _, again = run(lctx, x, y, 33)
        for n in first:
            assert torch.equal(torch.nan_to_num(first[n]), torch.nan_to_num(again[n])), n


def test_captured_pass_with_new_inputs(lctx):
    """Statistics, a teacher's entries from them, distillation and the gradient of the caller's own objective in one
    graph: its second replay has other logits."""
    T, V, k = 40, 3001, 16
    x, y = make(T, V, "f16", 1)
    other, _ = make(T, V, "f16", 2)
    xd, yd = x.cuda(), y.cuda()
    n = int((y >= 0).sum())
    f = lambda *s: torch.zeros(*s, device="cuda")  # noqa: E731
    logp, entropy, saved, top, result = f(T), f(T), f(T, 3), f(T, k), f(4)
    ids = torch.zeros(T, k, dtype=torch.int32, device="cuda")
    d, dd, scale = torch.zeros_like(xd), torch.zeros_like(xd), torch.tensor([256.0], device="cuda")
    ga, gb = f(T), f(T)

    def step():
        tl.tl_token_stats(lctx, xd, targets=yd, logp=logp, entropy=entropy, saved=saved, top_ids=ids, top_logp=top)
        ga.copy_(-(logp.exp()) / n)
        gb.fill_(0.01 / n)
        tl.tl_token_grad(lctx, xd, saved, d, targets=yd, grad_logp=ga, grad_entropy=gb, seed=scale)
        tl.tl_distill_loss(lctx, xd, top, ids, n, result, targets=yd, temperature=2.0, seed=scale, dlogits=dd)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for values in (x, other):
        xd.copy_(values)
        graph.replay()
        torch.cuda.synchronize()
        want = R.stats(values, y, k)
        compare({"logp": logp.cpu(), "entropy": entropy.cpu(), "saved": saved.cpu(), "ids": ids.cpu().long(), "top": top.cpu()}, want)
        replayed = d.clone(), dd.clone(), result.clone()
        step()
        for a, b in zip(replayed, (d, dd, result)):
            assert torch.equal(a, b)
        assert float(result[1]) >= 0 and float(result[3]) == n


def test_two_streams_at_once(lctx):
    """Calls that overlap share nothing: two streams, one context each, eight calls in turns."""
    other = tl.tl_loss_create(20000)
    cases = [(make(500, 20001, "bf16", i), ctx, torch.cuda.Stream()) for i, ctx in enumerate((lctx, other))]
    want, outs = [R.stats(x[:6], y[:6], 30) for (x, y), _, _ in cases], []
    held = [(x.cuda(), y.cuda()) for (x, y), _, _ in cases]
    torch.cuda.synchronize()
    for _ in range(4):
        for (xd, yd), (_, ctx, stream) in zip(held, cases):
            with torch.cuda.stream(stream):
                ids, top = torch.empty(500, 30, dtype=torch.int32, device="cuda"), torch.empty(500, 30, device="cuda")
                e, saved, lp = torch.empty(500, device="cuda"), torch.empty(500, 3, device="cuda"), torch.empty(500, device="cuda")
                tl.tl_token_stats(ctx, xd, yd, logp=lp, entropy=e, saved=saved, top_ids=ids, top_logp=top)
                outs.append((lp, e, saved, ids, top))
    torch.cuda.synchronize()
    for i, (lp, e, saved, ids, top) in enumerate(outs):
        compare({"logp": lp[:6].cpu(), "entropy": e[:6].cpu(), "saved": saved[:6].cpu(), "ids": ids[:6].cpu().long(),
                 "top": top[:6].cpu()}, want[i % 2])
        for a, b in zip(outs[i], outs[i % 2]):
            assert torch.equal(torch.nan_to_num(a), torch.nan_to_num(b))


def test_offsets_beyond_32_bits(lctx):
    """Rows 2^29 elements apart: the last starts at element 2^32."""
    T, V, ld = 9, 20000, 1 << 29
    free, _ = torch.cuda.mem_get_info()
    if free < 2 * (T * ld) + (1 << 30):
        pytest.skip("not enough memory")
    buf = torch.empty((T - 1) * ld + V, dtype=torch.bfloat16, device="cuda")
    X = torch.as_strided(buf, (T, V), (ld, 1))
    x, y = make(T, V, "bf16", 19, masked=0.0)
    X.copy_(x)
    ids, top = torch.zeros(T, 9, dtype=torch.int64, device="cuda"), torch.zeros(T, 9, device="cuda")
    e, saved = torch.zeros(T, device="cuda"), torch.zeros(T, 3, device="cuda")
    tl.tl_token_stats(lctx, X, entropy=e, saved=saved, top_ids=ids, top_logp=top)
    want = R.stats(x, None, 9)
    compare({"entropy": e.cpu(), "saved": saved.cpu(), "ids": ids.cpu(), "top": top.cpu()}, want)
    ga = torch.ones(T, device="cuda")
    tl.tl_token_grad(lctx, X, saved, X, targets=y.cuda(), grad_logp=ga)
    d = R.grad(x, y, torch.ones(T))
    assert ((X.cpu().double() - d).abs() <= d.abs() * 2.0 ** -8 * 1.01 + 1e-4).all()


@pytest.mark.parametrize("rows", [1, 200])
@pytest.mark.parametrize("V", [900, 20000, 40000])
def test_nearly_constant_fp32_rows(lctx, rows, V):
    """Thousands of entries within a few last places of each other: their order is still exact."""
    g = torch.Generator().manual_seed(V)
    base = (torch.full((3, V), 1000.0).view(torch.int32) + torch.randint(0, 40, (3, V), generator=g).int()).view(torch.float32)
    base[1] = -base[1]
    x = base[torch.arange(rows) % 3]
    _, got = run(lctx, x, None, 50)
    compare(got, {n: v[torch.arange(rows) % 3] for n, v in R.stats(base, None, 50).items()})


def test_one_row_into_wider_buffers(lctx):
    x, y = make(1, 3000, "bf16", 3)
    ids, top = torch.full((4, 20), 7, dtype=torch.int32, device="cuda"), torch.full((4, 9), 7.0, device="cuda")
    tl.tl_token_stats(lctx, x.cuda(), top_ids=ids[1:2, :5], top_logp=top[2:3, :5])
    want = R.stats(x, None, 5)
    assert torch.equal(ids[1, :5].cpu().long(), want["ids"][0]) and (ids[1, 5:] == 7).all() and (ids[[0, 2, 3]] == 7).all()
    close(top[2:3, :5].cpu(), want["top"], REL + 4 * EPS * want["top"].abs(), "top")
    assert (top[2, 5:] == 7).all() and (top[[0, 1, 3]] == 7).all()
