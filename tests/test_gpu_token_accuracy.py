"""How far row statistics are from fp64, over many rows, in units that the kernels' corrections show in.

u = 2^-24 / sqrt(3) = 3.44e-8 is the rms of one rounding to fp32, of a value next to a power of two from above (the worst)."""
import math

import pytest

torch = pytest.importorskip("torch")

import loss_scaled_adamw_gb300 as tl
import test_gpu_token as G

pytestmark = pytest.mark.gpu

lctx = G.lctx
DT = G.DT
U = 2.0 ** -24 / math.sqrt(3)


def statistics(lctx, x, y, tau=1.0, k=0):
    T = x.shape[0]
    lp, e, saved = torch.zeros(T, device="cuda"), torch.zeros(T, device="cuda"), torch.zeros(T, 3, device="cuda")
    kw = dict(top_ids=torch.zeros(T, k, dtype=torch.int32, device="cuda"), top_logp=torch.zeros(T, k, device="cuda")) if k else {}
    tl.tl_token_stats(lctx, x, targets=y, logp=lp, entropy=e, saved=saved, temperature=tau, **kw)
    return lp.double(), e.double(), kw.get("top_logp")


def exact(x, y, it):
    """log q of the labels, entropy, log of the sum against the largest, and sqrt(sum q^2 (log q + H)^2), at 1 / temperature it."""
    out = []
    for a in range(0, x.shape[0], 64):
        z = x[a:a + 64].double() * it
        lsm = torch.log_softmax(z, 1)
        q = lsm.exp()
        h = -(q * lsm).sum(1)
        shown = (q * (lsm + h[:, None])).square().sum(1).sqrt()
        out.append(torch.stack([lsm.gather(1, y[a:a + 64, None])[:, 0], h, -lsm.max(1).values, shown]))
    return torch.cat(out, 1)


def rows(T, V, dtype, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = (torch.randn(T, V, generator=g, device="cuda") * 2.5).to(DT[dtype])
    return x, torch.randint(0, V, (T,), generator=g, device="cuda")


def rms(v):
    return float(v.square().mean().sqrt())


FORMS = [(2048, 1000, "bf16", 0), (2048, 1000, "f16", 8), (2048, 8192, "bf16", 8), (2048, 8192, "f32", 0), (512, 50001, "bf16", 20),
         (512, 50001, "f32", 20), (512, 128256, "bf16", 0), (512, 128256, "f16", 64), (512, 126599, "f32", 0), (19, 128256, "bf16", 20)]


@pytest.mark.parametrize("T,V,dtype,k", FORMS)
def test_log_probabilities_are_rounded_once(lctx, T, V, dtype, k):
    """Rounding the result has the rms q of the exact values.  The logarithm of the sum adds at most 2e-7: the exponential's
    error (2^-22, as if one term made the sum: 1.4e-7), eight partial sums (sqrt(8) u = 1e-7), log2's last place (0.4e-7).
    16-bit rows take log2 e in fp32, off by 1.34e-8 of itself, times x_y - E_q[x], whose mean is the variance 6.25:
    0.84e-7; with the exponential's mean error of 2^-24 the mean is held to 1.5e-7."""
    x, y = rows(T, V, dtype, V + k)
    lp, _, _ = statistics(lctx, x, y, 1.0, k)
    want = exact(x, y, 1.0)[0]
    e, q = lp - want, rms(want.float().double() - want)
    bound = math.sqrt(q * q + 2e-7 ** 2) * (1 + 5 / math.sqrt(2 * T))
    assert rms(e - e.mean()) <= bound, (rms(e - e.mean()), bound)
    assert abs(float(e.mean())) <= 1.5e-7 + 5 * bound / math.sqrt(T), float(e.mean())


@pytest.mark.parametrize("T,V,dtype,k", FORMS)
def test_entropies(lctx, T, V, dtype, k):
    """H = log S + D, D = sum q (max - x): log S and the sum are rounded once each (u log S, u H); D, the quotient of two
    sums, by at most 20 partial sums and products of its size (sqrt(20) u D), S by sqrt(9) u.  A term whose exponent of
    up to 16 bits rounds by 2^-21 (0.69 * 2.75e-7 = 1.9e-7) and whose exponential is off by 1.4e-7 moves H by
    q (log q + H) times 2.4e-7.  The scale's rounding, which only 16-bit rows leave, moves all rows one way."""
    x, y = rows(T, V, dtype, 3 * V + k)
    _, got, _ = statistics(lctx, x, y, 1.0, k)
    _, want, log_sum, shown = exact(x, y, 1.0)
    d = want - log_sum
    each = (U * (log_sum ** 2 + want ** 2 + 20 * d ** 2 + 9).sqrt()).square() + (2.4e-7 * shown).square()
    bound = float(each.mean().sqrt()) * (1 + 5 / math.sqrt(2 * T))
    e = got - want
    assert rms(e - e.mean()) <= bound, (rms(e - e.mean()), bound)
    at_rounded = exact(x, y, float(torch.tensor(1.4426950408889634)) * math.log(2))[1]
    drift = 0.0 if dtype == "f32" else abs(float((at_rounded - want).mean()))
    assert abs(float(e.mean())) <= drift + 2.0 ** -24 * 1.5 + 5 * bound / math.sqrt(T), (float(e.mean()), drift)


@pytest.mark.parametrize("V,k", [(126599, 0), (50001, 8), (2100, 8)])
def test_scale_of_fp32_rows_is_not_rounded(lctx, V, k):
    """Entropies at the scale log2 e / 0.72 rounded to fp32 (by 5e-8 of it) are off by B in the mean; the kernel carries
    the rest of the scale, so its mean is within a third of B (S's mean error of 2^-24 is far below that)."""
    T, tau = 512, 0.72
    x, y = rows(T, V, "f32", V)
    _, got, _ = statistics(lctx, x, y, tau, k)
    tau32 = float(torch.tensor(tau))
    want = exact(x, y, 1 / tau32)[1]
    rounded = float(torch.tensor(1.4426950408889634 / tau32, dtype=torch.float64).float())
    B = float((exact(x, y, rounded * math.log(2))[1] - want).mean())
    assert abs(B) > 2e-7
    assert abs(float((got - want).mean())) < abs(B) / 3, (float((got - want).mean()), B)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T,k", [(1024, 0), (1024, 8), (64, 8), (64, 0)])
def test_a_token_that_makes_the_sum(lctx, T, k, dtype):
    """A thread meets zeros first and the label, 16 to 31 bits above them, later: against the zeros the label's exponent
    rounds to 2^-20 (rms 5.5e-7, times ln 2: 3.8e-7 of the sum), beside the exponential's 2^-22.  Taken again in full it
    has two roundings, the sums above it ten, log2 one: sqrt(13) u = 1.25e-7 in the rms."""
    V = 128256
    g = torch.Generator(device="cuda")
    g.manual_seed(T + k)
    x = torch.full((T, V), -200.0, device="cuda")
    x[:, :V // 4] = 0.0
    y = torch.randint(V // 2, V, (T,), generator=g, device="cuda")
    x[torch.arange(T, device="cuda"), y] = 11.2 + 10 * torch.rand(T, generator=g, device="cuda")
    x = x.to(DT[dtype])
    lp, _, _ = statistics(lctx, x, y, 1.0, k)
    e = lp - exact(x, y, 1.0)[0]
    assert rms(e) <= math.sqrt(13) * U * (1 + 5 / math.sqrt(2 * T)), rms(e)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gradient_of_rows_far_apart(lctx, dtype):
    """Rows 2^29 elements apart have the gradients, bit for bit, that they have side by side."""
    T, V, ld = 9, 20000, 1 << 29
    free, _ = torch.cuda.mem_get_info()
    if free < DT[dtype].itemsize * T * ld + (1 << 30):
        pytest.skip("not enough memory")
    x, y = G.make(T, V, dtype, 23, masked=0.0)
    x, y = x.cuda(), y.cuda()
    saved, near = torch.zeros(T, 3, device="cuda"), torch.zeros_like(x)
    tl.tl_token_stats(lctx, x, saved=saved)
    a, b = torch.linspace(-1, 2, T, device="cuda"), torch.linspace(1, -1, T, device="cuda")
    tl.tl_token_grad(lctx, x, saved, near, targets=y, grad_logp=a, grad_entropy=b)
    assert (near != 0).all(1).all() or dtype == "bf16"
    far = torch.as_strided(torch.empty((T - 1) * ld + V, dtype=x.dtype, device="cuda"), (T, V), (ld, 1))
    far.copy_(x)
    tl.tl_token_grad(lctx, far, saved, far, targets=y, grad_logp=a, grad_entropy=b)
    assert torch.equal(far, near)
