"""Plain fp64 statements of the objectives over logits (CPU, torch), for the tests.

Every function takes the logits as given (any float type, converted exactly) and returns
fp64: the loss of each row or pair, the mean terms, and the gradient of the mean loss
with respect to the logits by the written formula.  `checked_logits` in the CPU tests
holds the formulas against central differences.
"""
import math

import torch

NAN = float("nan")


def _softmax(x, tau):
    z = x.double() / tau
    m = z.amax(1, keepdim=True)
    e = torch.exp(z - m)
    s = e.sum(1, keepdim=True)
    return z - m - torch.log(s), e / s      # log q, q


def logprob(x, y, tau=1.0):
    """Log-probabilities of the targets; 0 for ignored rows, NaN for a target beyond the vocabulary."""
    V = x.shape[1]
    out = torch.zeros(x.shape[0], dtype=torch.float64)
    for t, j in enumerate(y.tolist()):
        if j >= 0:
            out[t] = _softmax(x[t:t + 1], tau)[0][0, j] if j < V else NAN
    return out


def _row_gradient(x, y, g, tau, factor):
    """factor / tau * g_t * (1[j = y] - q_j) per valid row, zero elsewhere."""
    d = torch.zeros(x.shape, dtype=torch.float64)
    for t, j in enumerate(y.tolist()):
        if j < 0:
            continue
        if j >= x.shape[1]:
            d[t] = NAN
            continue
        q = _softmax(x[t:t + 1], tau)[1][0]
        one = torch.zeros_like(q)
        one[j] = 1.0
        d[t] = factor / tau * g[t] * (one - q)
    return d


def policy(x, y, old, adv, n, ref=None, clip_low=0.2, clip_high=0.2, kl_weight=0.0, tau=1.0, seed=1.0):
    T = x.shape[0]
    lp = logprob(x, y, tau)
    loss, sur, kl, g = (torch.zeros(T, dtype=torch.float64) for _ in range(4))
    for t in range(T):
        if y[t] < 0:
            continue
        A, l = float(adv[t]), float(lp[t])
        r = math.exp(l - float(old[t]))
        held = min(max(r, 1 - clip_low), 1 + clip_high) * A
        sur[t] = -min(r * A, held) if r == r else NAN
        g[t] = -r * A if r * A <= held or r != r else 0.0
        if ref is not None:
            d = float(ref[t]) - l
            kl[t] = math.exp(d) - d - 1
            if kl_weight > 0:
                g[t] += kl_weight * (1 - math.exp(d))
        loss[t] = sur[t] + (kl_weight * kl[t] if kl_weight > 0 else 0.0)
    res = torch.tensor([loss.sum() / n, sur.sum() / n, kl.sum() / n, float((y >= 0).sum())])
    return {"logp": lp, "loss": loss, "result": res, "dx": _row_gradient(x, y, g, tau, seed / n), "g": g}


def preference(x, y, seq, n, ref=None, beta=0.1, smooth=0.0, tau=1.0, seed=1.0):
    T = x.shape[0]
    lp = logprob(x, y, tau)
    ratio = lp.clone()
    if ref is not None:
        ratio = torch.where(y >= 0, lp - ref.double(), 0.0)
    s = [min(max(int(v), 0), T) for v in seq]
    pairs = len(s) // 2
    loss, reward, g = torch.zeros(pairs).double(), torch.zeros(2 * pairs).double(), torch.zeros(T).double()
    margin, won = 0.0, 0
    for p in range(pairs):
        c, r = ratio[s[2 * p]:s[2 * p + 1]].sum().item(), ratio[s[2 * p + 1]:s[2 * p + 2]].sum().item()
        h = beta * (c - r)
        up, down = (math.log1p(math.exp(-abs(h))) - min(v, 0.0) for v in (h, -h))   # -log sg(h), -log sg(-h)
        loss[p] = (1 - smooth) * up + smooth * down
        dh = -beta * ((1 - smooth) * math.exp(-down) - smooth * math.exp(-up))
        g[s[2 * p]:s[2 * p + 1]], g[s[2 * p + 1]:s[2 * p + 2]] = dh, -dh
        reward[2 * p], reward[2 * p + 1] = beta * c, beta * r
        margin, won = margin + h, won + (h > 0)
    res = torch.tensor([float(loss.sum()) / n, margin / n, won / n, float(pairs)])
    return {"logp": lp, "loss": loss, "reward": reward, "result": res, "g": g,
            "dx": _row_gradient(x, y, g, tau, seed / n)}


def distill(x, teacher, ids, n, y=None, kd_weight=1.0, ce_weight=0.0, tau=1.0, seed=1.0):
    T, V = x.shape
    loss, kds, ces = (torch.zeros(T, dtype=torch.float64) for _ in range(3))
    dx = torch.zeros(T, V, dtype=torch.float64)
    valid = 0
    for t in range(T):
        j = -1 if y is None else int(y[t])
        if y is not None and j < 0:
            continue
        valid += 1
        use = [] if teacher is None or kd_weight == 0 else [i for i, v in enumerate(ids[t].tolist()) if v >= 0]
        if j >= V or any(int(ids[t, i]) >= V for i in use):
            loss[t], dx[t] = NAN, NAN
            kds[t] = NAN
            ces[t] = NAN if ce_weight > 0 else 0.0
            continue
        if use:
            logits = teacher[t, use].double() / tau
            if logits.max() > -math.inf:
                logp = logits - torch.logsumexp(logits, 0)
                p = torch.exp(logp)
                logq, q = (v[0] for v in _softmax(x[t:t + 1], tau))
                at = ids[t, use].long()
                on = p > 0
                kds[t] = tau ** 2 * (p[on] * (logp[on] - logq[at][on])).sum()
                full = torch.zeros(V, dtype=torch.float64).index_add_(0, at, p)
                dx[t] += seed / n * kd_weight * tau * (q - full)
                loss[t] += kd_weight * kds[t]
        if ce_weight > 0:
            logq, q = (v[0] for v in _softmax(x[t:t + 1], 1.0))
            ces[t] = -logq[j]
            one = torch.zeros(V, dtype=torch.float64)
            one[j] = 1.0
            dx[t] += seed / n * ce_weight * (q - one)
            loss[t] += ce_weight * ces[t]
    res = torch.tensor([loss.sum() / n, kds.sum() / n, ces.sum() / n, float(valid)])
    return {"loss": loss, "result": res, "dx": dx, "kd": kds}
