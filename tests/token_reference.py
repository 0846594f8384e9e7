"""Plain fp64 statements of the row statistics, their gradient and dropout, for the tests."""
import math

import numpy as np
import torch

NAN, INF = float("nan"), float("inf")


def stats(x, y=None, k=0, tau=1.0):
    """Per row: logp, entropy, saved [max, log_sum, entropy], ids and top [k] in fp64."""
    T, V = x.shape
    out = {"logp": torch.zeros(T, dtype=torch.float64), "entropy": torch.zeros(T, dtype=torch.float64),
           "saved": torch.zeros(T, 3, dtype=torch.float64), "ids": torch.full((T, k), -1, dtype=torch.int64),
           "top": torch.zeros(T, k, dtype=torch.float64)}
    for t in range(T):
        j = 0 if y is None else int(y[t])
        if j < 0:
            continue
        row = x[t].double()
        m = row.max() if not torch.isnan(row).any() else torch.tensor(NAN)
        if not math.isfinite(m):                      # NaN, +inf, or nothing but -inf
            out["logp"][t] = out["entropy"][t] = NAN
            out["saved"][t] = out["top"][t] = NAN
            continue
        z = (row - m) / tau
        e = torch.exp(z)
        log_sum = torch.log(e.sum())
        log_q = z - log_sum
        q = e / e.sum()
        entropy = -(q * torch.where(q > 0, log_q, torch.zeros_like(q))).sum()
        out["logp"][t] = log_q[j] if j < V else NAN
        out["entropy"][t] = entropy
        out["saved"][t] = torch.stack([m, log_sum, entropy])
        order = torch.sort(row, descending=True, stable=True).indices[:k].tolist()
        out["top"][t] = -INF
        for i, v in enumerate(v for v in order if row[v] > -INF):
            out["ids"][t, i], out["top"][t, i] = v, log_q[v]
    return out


def grad(x, y=None, ga=None, gb=None, tau=1.0, seed=1.0):
    """seed * d/dx sum_t ga_t logp_t + gb_t entropy_t by the written formula."""
    T, V = x.shape
    d = torch.zeros(x.shape, dtype=torch.float64)
    for t in range(T):
        j = 0 if y is None else int(y[t])
        if j < 0:
            continue
        m, log_sum, entropy = stats(x[t:t + 1], None, 0, tau)["saved"][0]
        if not math.isfinite(m) or j >= V:
            d[t] = NAN
            continue
        log_q = (x[t].double() - m) / tau - log_sum
        q = torch.exp(log_q)
        a, b = (0.0 if g is None else float(g[t]) for g in (ga, gb))
        d[t] = -a * q - b * q * torch.where(q > 0, log_q + entropy, torch.zeros_like(q))
        if ga is not None:
            d[t, j] += a
    return d * seed / tau


MASK = 0xFFFFFFFF


def philox(counter, key):
    """Philox4x32-10 on Python integers: the four words of one counter."""
    c, (k0, k1) = list(counter), key
    for _ in range(10):
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [(b >> 32) ^ c[1] ^ k0, b & MASK, (a >> 32) ^ c[3] ^ k1, a & MASK]
        k0, k1 = (k0 + 0x9E3779B9) & MASK, (k1 + 0xBB67AE85) & MASK
    return c


def numbers(first, count, seed, ticket, site):
    """The 16-bit numbers of elements first .. first + count - 1 (numpy, 64-bit unsigned)."""
    seed, u = seed % 2 ** 64, np.uint64
    at = np.arange(first // 8, (first + count + 7) // 8, dtype=u)
    c = [at & u(MASK), (at >> u(32)) | u((ticket >> 32) << 8), np.full_like(at, ticket & MASK), np.full_like(at, site)]
    k0, k1 = seed & MASK, seed >> 32
    for _ in range(10):
        a, b = c[0] * u(0xD2511F53), c[2] * u(0xCD9E8D57)
        c = [(b >> u(32)) ^ c[1] ^ u(k0), b & u(MASK), (a >> u(32)) ^ c[3] ^ u(k1), a & u(MASK)]
        k0, k1 = (k0 + 0x9E3779B9) & MASK, (k1 + 0xBB67AE85) & MASK
    halves = np.stack([h for w in c for h in (w & u(0xFFFF), w >> u(16))], 1).reshape(-1)
    return halves[first % 8:first % 8 + count].astype(np.int64)


def dropout(x, p, seed, ticket, site, residual=None):
    """fp64; x is of any shape, taken row-major."""
    limit = round(p * 65536)
    keep = torch.from_numpy(numbers(0, x.numel(), seed, ticket, site) >= limit).view(x.shape)
    y = torch.where(keep, x.double() / max(1 - limit / 65536, 2.0 ** -17), torch.zeros((), dtype=torch.float64))
    return y if residual is None else y + residual.double()
