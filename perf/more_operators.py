"""Statistics of vocabulary logits, their gradient, and dropout as measured work: cases, inputs, plain forms, exact values.

Each case is one call of tl_token_stats, tl_token_grad or tl_dropout.  `run` computes it
in its plain form (elementary torch operations in fp32, rounded once at the end) or, with
`own` set, through the library.  `exact` gives the same outputs from the definition in
fp64: the gradients by automatic differentiation, the alternatives by a stable sort, the
random bits by products of 16-bit halves.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
IGNORED = -100

# 4,096 rows are the 8 x 512 positions of a micro-batch; 128,256 and 8,192 entries the vocabularies,
# 2,048 and 288 the widths, 8,192 and 768 the inner widths of the llama_1b and llama_10m workloads.
# 50,001 and 32,003 are odd vocabularies, whose rows start at every element phase.
ROWS, VOCAB, VOCAB_SMALL, VOCAB_ODD = 4096, 128256, 8192, 50001
WIDTH, INNER = 2048, 8192
MOST_BYTES = 2 * ROWS * VOCAB * 2            # a pass over the largest case: logits in, gradients out


def listed():
    return [
        # the one token just sampled with the large vocabulary, its entropy and twenty alternatives: latency
        _stats("stats_one_token", 1, VOCAB, "bf16", k=20),
        # a few short answers of the small model
        _stats("stats_small", 64, VOCAB_SMALL, "f16", k=5, masked=0.125),
        # fp32 logits of an odd vocabulary at a sampling temperature, 64-bit ids, padded vocabulary entries excluded
        _stats("stats_odd_f32", 777, VOCAB_ODD, "f32", tau=0.7, k=8, masked=0.3, wide_ids=True, excluded=True),
        # a teacher's 64 likeliest entries for a whole micro-batch, as distillation takes them
        _stats("stats_teacher_llama_1b", ROWS, VOCAB, "bf16", k=64, masked=0.125),
        # the training forward of an objective over log-probabilities and entropies: no alternatives
        _stats("stats_llama_1b", ROWS, VOCAB, "bf16", masked=0.125),
        # the gradient for a few short answers of the small model
        _grad("grad_small", 64, VOCAB_SMALL, "f16", masked=0.125),
        # entropies alone, odd vocabulary, fp32
        _grad("grad_odd_f32", 1500, 32003, "f32", tau=0.7, masked=0.1, first=False, excluded=True),
        # the gradient for a whole micro-batch of the large model
        _grad("grad_llama_1b", ROWS, VOCAB, "bf16", masked=0.125),
        # one token's hidden state (a short rollout in training mode): latency
        _dropout("dropout_one_token", 1, WIDTH, "bf16", 0.1),
        # columns cut out of a wider fp32 matrix, odd sizes: neither rows nor elements at a common phase
        _dropout("dropout_odd_f32", 3001, 1153, "f32", 0.25, residual=True, pad=6),
        # a residual branch of the large model over a micro-batch
        _dropout("dropout_residual_llama_1b", ROWS, WIDTH, "bf16", 0.1, residual=True),
        # the inner activations of all eight micro-batches of an update, backwards: the gradient through the mask
        _dropout("dropout_inner_llama_1b", 8 * ROWS, INNER, "bf16", 0.1, backward=True),
    ]


def _stats(name, rows, vocab, dtype, tau=1.0, k=0, masked=0.0, wide_ids=False, excluded=False):
    return {"name": name, "op": "stats", "rows": rows, "vocab": vocab, "dtype": dtype, "tau": tau, "k": k,
            "masked": masked, "wide_ids": wide_ids, "excluded": excluded}


def _grad(name, rows, vocab, dtype, tau=1.0, masked=0.0, first=True, second=True, excluded=False):
    return {"name": name, "op": "grad", "rows": rows, "vocab": vocab, "dtype": dtype, "tau": tau, "masked": masked,
            "first": first, "second": second, "excluded": excluded}


def _dropout(name, rows, cols, dtype, p, residual=False, pad=0, backward=False):
    return {"name": name, "op": "dropout", "rows": rows, "cols": cols, "dtype": dtype, "p": p, "residual": residual,
            "pad": pad, "backward": backward}


def draw(rng):
    log = lambda lo, hi: int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))  # noqa: E731
    op = rng.choice(["stats", "stats", "grad", "dropout"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    size = 4 if dtype == "f32" else 2
    if op == "dropout":
        cols, rows = log(64, INNER), log(1, 8 * ROWS)
        if rng.random() < 0.7:
            cols = max(64, cols // 32 * 32)
        c = _dropout("", rows, cols, dtype, rng.choice([0.05, 0.1, 0.3, 0.5]), rng.random() < 0.5,
                     rng.choice([0, 0, 0, 7, 64]), rng.random() < 0.3)
        c["residual"] = c["residual"] and not c["backward"]
        c["rows"] = max(1, min(rows, MOST_BYTES // ((3 if c["residual"] else 2) * size * cols)))
        del c["name"]
        return c
    vocab = log(500, VOCAB)
    if rng.random() < 0.5:
        vocab = max(512, vocab // 64 * 64)          # half of them padded to a round size, the rest as they come
    rows = min(log(1, 4 * ROWS), max(1, MOST_BYTES // (2 * size * vocab)))
    common = dict(tau=rng.choice([1.0, 1.0, 0.7, 2.0]), masked=rng.choice([0.0, 0.125, 0.4]), excluded=rng.random() < 0.3)
    if op == "stats":
        k = 0 if rng.random() < 0.2 else min(log(1, 256), vocab)
        c = _stats("", rows, vocab, dtype, k=k, wide_ids=rng.random() < 0.3, **common)
    else:
        which = rng.choice([(True, True), (True, True), (True, False), (False, True)])
        c = _grad("", rows, vocab, dtype, first=which[0], second=which[1], **common)
    del c["name"]
    return c


def _mask(case):
    """The ignored rows (the same for every seed): the padded end of each 512-row sequence."""
    ignored = [False] * case["rows"]
    for at in range(0, case["rows"], 512):
        n = min(512, case["rows"] - at)
        for i in range(at + n - int(n * case["masked"]), at + n):
            ignored[i] = True
    return ignored


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (_prepare_dropout if case["op"] == "dropout" else _prepare_rows)(case, seed, g)


def _prepare_rows(case, seed, g):
    T, V, dev = case["rows"], case["vocab"], "cuda"
    s = {"case": dict(case)}
    # logits of a language model: a broad spread, the label among the likely entries
    target = torch.randint(0, V - V // 64, (T,), generator=g, device=dev)
    x = torch.randn(T, V, generator=g, device=dev) * 2.5
    x[torch.arange(T, device=dev), target] += 2 + 12 * torch.rand(T, generator=g, device=dev)
    if case["excluded"]:
        x[:, V - V // 64:] = float("-inf")           # entries that pad the vocabulary
    s["x"] = x = x.to(DTYPES[case["dtype"]])
    s["target"] = torch.where(torch.tensor(_mask(case), device=dev), IGNORED, target)
    if case["op"] == "stats":
        s["logp"], s["entropy"] = torch.zeros(T, device=dev), torch.zeros(T, device=dev)
        s["saved"] = torch.zeros(T, 3, device=dev)
        if case["k"]:
            s["ids"] = torch.zeros(T, case["k"], dtype=torch.int64 if case["wide_ids"] else torch.int32, device=dev)
            s["top"] = torch.zeros(T, case["k"], device=dev)
        return s
    # what the forward has saved of each row, and the gradients of an objective of the user's own: a mean
    # over valid rows of a policy term and of an entropy bonus
    valid = max(1, T - sum(_mask(case)))
    s["saved"] = torch.empty(T, 3, device=dev)
    for a in range(0, T, 512):
        z = x[a:a + 512].double()
        m = z.amax(1, keepdim=True)
        w = (z - m) / case["tau"]
        log_sum = torch.logsumexp(w, 1)
        q = torch.softmax(w, 1)
        entropy = log_sum - (q * w.clamp(min=-1e300)).sum(1)
        s["saved"][a:a + 512] = torch.stack([m[:, 0], log_sum, entropy], 1).float()
    s["ga"] = torch.randn(T, generator=g, device=dev) / valid if case["first"] else None
    s["gb"] = torch.randn(T, generator=g, device=dev) * (0.5 / valid) if case["second"] else None
    s["scale"] = torch.full((1,), 2.0 ** 14 if case["dtype"] == "f16" else 1.0, device=dev)
    s["dx"] = torch.empty_like(x)
    return s


def _prepare_dropout(case, seed, g):
    T, C, P, dt = case["rows"], case["cols"], case["pad"], DTYPES[case["dtype"]]

    def matrix():
        return torch.randn(T, C + P, generator=g, device="cuda").to(dt)[:, P // 2:P // 2 + C]

    s = {"case": dict(case), "x": matrix(), "r": matrix() if case["residual"] else None}
    s["y"] = torch.empty(T, C + P, dtype=dt, device="cuda")[:, P // 2:P // 2 + C]
    # the run's seed, and the ticket of this micro-batch
    s["key"] = torch.tensor([0x5EED0000 + 977 * seed, 3 * seed + 1], dtype=torch.int64, device="cuda")
    s["site"] = 2 * (seed % 97) + 1
    return s


def run(state):
    if own:
        return _own(state)
    return {"stats": _plain_stats, "grad": _plain_grad, "dropout": _plain_dropout}[state["case"]["op"]](state)


def _plain_stats(s):
    c, x, tau = s["case"], s["x"], s["case"]["tau"]
    valid = s["target"] >= 0
    x32 = x.float()
    m = x32.amax(1, keepdim=True)
    z = (x32 - m) / tau
    e = z.exp()
    total = e.sum(1, keepdim=True)
    log_sum = total.log()
    logp = torch.where(valid, (z.gather(1, s["target"].clamp(min=0)[:, None]) - log_sum)[:, 0], 0.0)
    entropy = torch.where(valid, (log_sum - (e * z.clamp_(min=-1e30)).sum(1, keepdim=True) / total)[:, 0], 0.0)
    saved = torch.where(valid[:, None], torch.stack([m[:, 0], log_sum[:, 0], entropy], 1), 0.0)
    out = {"logp": logp, "entropy": entropy, "saved": saved}
    del z, e
    if c["k"]:
        # keys that no two entries share: the logit's order, then the lower id
        low = 0xFFFFFFFF - torch.arange(c["vocab"], device=x.device)
        best = []
        for a in range(0, c["rows"], 1024):
            bits = (x32[a:a + 1024] + 0.0).view(torch.int32).long()
            order = torch.where(bits < 0, -(bits & 0x7FFFFFFF), bits)
            best.append(0xFFFFFFFF - (order * 2 ** 32 + low).topk(c["k"], 1).values.bitwise_and(0xFFFFFFFF))
        ids = torch.cat(best)
        top = (x32.gather(1, ids) - m) / tau - log_sum
        ids = torch.where(top == float("-inf"), -1, ids)
        out["top"] = torch.where(valid[:, None], top, 0.0)
        out["ids"] = torch.where(valid[:, None], ids, -1).to(s["ids"].dtype)
    return out


def _plain_grad(s):
    c, x, it = s["case"], s["x"], 1.0 / s["case"]["tau"]
    valid = (s["target"] >= 0)[:, None]
    m, log_sum, entropy = (s["saved"][:, i:i + 1] for i in range(3))
    log_q = (x.float() - m) * it - log_sum
    q = log_q.exp()
    factor = torch.zeros_like(m)
    if c["second"]:
        factor = s["gb"][:, None] * (log_q.clamp_(min=-1e30) + entropy)
    if c["first"]:
        factor = factor + s["ga"][:, None]
    d = q.mul_(-it * s["scale"] * factor)
    if c["first"]:
        d.scatter_add_(1, s["target"].clamp(min=0)[:, None], (it * s["scale"] * s["ga"])[:, None])
    return {"dx": d.masked_fill_(~valid, 0.0).to(x.dtype)}


LOW32 = 0xFFFFFFFF


def _philox(c, k):
    for i in range(10):
        p0, p1 = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57        # 64-bit products, kept modulo 2^64
        c = [((p1 >> 32) & LOW32) ^ c[1] ^ k[0], p1 & LOW32, ((p0 >> 32) & LOW32) ^ c[3] ^ k[1], p0 & LOW32]
        k = [(k[0] + 0x9E3779B9) & LOW32, (k[1] + 0xBB67AE85) & LOW32]
    return c


def _keep(numel, p, key, site):
    """Which of the elements are kept: 16 bits each, eight to a block of the generator."""
    threshold, seed, ticket = int(round(p * 65536)), key[0], key[1]
    keep = torch.empty((numel + 7) // 8, 8, dtype=torch.bool, device=key.device)
    for a in range(0, keep.shape[0], 1 << 22):
        part = keep[a:a + (1 << 22)]
        at = torch.arange(a, a + part.shape[0], device=key.device)
        counter = [at & LOW32, (at >> 32) | ((ticket >> 32) << 8), torch.zeros_like(at) + (ticket & LOW32),
                   torch.full_like(at, site)]
        for i, w in enumerate(_philox(counter, [seed & LOW32, (seed >> 32) & LOW32])):
            part[:, 2 * i] = (w & 0xFFFF) >= threshold
            part[:, 2 * i + 1] = (w >> 16) >= threshold
    return keep.view(-1)[:numel], threshold / 65536


def _plain_dropout(s):
    c, x = s["case"], s["x"]
    keep, p = _keep(x.numel(), c["p"], s["key"], s["site"])
    y = torch.where(keep.view(x.shape), x.float() * (1 / (1 - p)), 0.0)
    if s["r"] is not None:
        y = y + s["r"].float()
    return {"y": y.to(x.dtype)}


_context = None


def _own(s):
    import loss_scaled_adamw_gb300 as tl
    global _context
    c, x = s["case"], s["x"]
    if c["op"] == "dropout":
        tl.tl_dropout(x, s["y"], c["p"], s["key"], site=s["site"], residual=s["r"])
        return {"y": s["y"]}
    if _context is None:      # one context for a process, as a trainer keeps it
        _context = tl.tl_loss_create(max_rows=4 * ROWS)
    if c["op"] == "grad":
        tl.tl_token_grad(_context, x, s["saved"], s["dx"], targets=s["target"], grad_logp=s["ga"],
                         grad_entropy=s["gb"], temperature=c["tau"], seed=s["scale"])
        return {"dx": s["dx"]}
    out = {"logp": s["logp"], "entropy": s["entropy"], "saved": s["saved"]}
    if c["k"]:
        out.update(top=s["top"], ids=s["ids"])
    tl.tl_token_stats(_context, x, targets=s["target"], logp=s["logp"], entropy=s["entropy"], top_ids=out.get("ids"),
                      top_logp=out.get("top"), saved=s["saved"], temperature=c["tau"])
    return out


def work(case):
    """Logits of the rows that carry loss read once, every gradient row written once, the row inputs and
    outputs; each activation read and written once.  Random bits cost operations and no bytes."""
    size = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "dropout":
        n = case["rows"] * case["cols"]
        return {"bytes": (3 if case["residual"] else 2) * n * size, "flops": 2 * n}
    T, V = case["rows"], case["vocab"]
    valid = T - sum(_mask(case))
    if case["op"] == "stats":
        return {"bytes": valid * V * size + 8 * T + T * (20 + case["k"] * (12 if case["wide_ids"] else 8)), "flops": 8 * valid * V}
    rows = 8 * T + valid * (12 + 4 * case["first"] + 4 * case["second"])
    return {"bytes": valid * V * size + T * V * size + rows, "flops": 8 * valid * V}


def _bits_by_halves(element, seed, ticket, site):
    """The 16 random bits of each element, the generator's products made of 16-bit halves."""
    def product(a, b):
        al, ah, bl, bh = a % 65536, a // 65536, b % 65536, b // 65536
        low, mid, other = al * bl, ah * bl, al * bh
        carry = (low // 65536 + mid % 65536 + other % 65536)
        return ah * bh + mid // 65536 + other // 65536 + carry // 65536, carry % 65536 * 65536 + low % 65536
    block = element // 8
    r0, r1 = block % 2 ** 32, block // 2 ** 32 + ticket // 2 ** 32 * 256
    r2, r3 = torch.full_like(block, ticket % 2 ** 32), torch.full_like(block, site)
    k0, k1 = seed % 2 ** 32, seed // 2 ** 32
    for _ in range(10):
        high0, low0 = product(r0, 0xD2511F53)
        high1, low1 = product(r2, 0xCD9E8D57)
        r0, r1, r2, r3 = high1 ^ r1 ^ k0, low1, high0 ^ r3 ^ k1, low0
        k0, k1 = (k0 + 0x9E3779B9) % 2 ** 32, (k1 + 0xBB67AE85) % 2 ** 32
    place = element % 8
    word = torch.stack([r0, r1, r2, r3]).gather(0, (place // 2)[None])[0]
    return torch.where(place % 2 == 1, word // 65536, word % 65536)


def exact(case, seed):
    """The definition in fp64, blocks of rows at a time; gradients by automatic differentiation."""
    s = prepare(case, seed)
    x = s["x"]
    if case["op"] == "dropout":
        seed64, ticket = s["key"].tolist()
        share = round(case["p"] * 65536) / 65536
        flat = torch.empty(x.numel(), dtype=torch.float64, device=x.device)
        x64 = x.reshape(-1)
        for a in range(0, x.numel(), 1 << 24):
            b = min(x.numel(), a + (1 << 24))
            bits = _bits_by_halves(torch.arange(a, b, device=x.device), seed64, ticket, s["site"])
            flat[a:b] = x64[a:b].double() / (1 - share) * (bits / 65536 >= share)
        y = flat.view(x.shape)
        return {"y": y if s["r"] is None else y + s["r"].double()}
    T, tau, ok = case["rows"], case["tau"], s["target"] >= 0
    block = max(1, (1 << 25) // case["vocab"])

    def logp_and_entropy(z, a, b):
        lsm = torch.nn.functional.log_softmax(z, dim=1)
        picked = lsm[torch.arange(b - a, device=x.device), s["target"][a:b].clamp(min=0)]
        finite = torch.where(torch.isinf(lsm), 0.0, lsm)
        return picked, -(lsm.exp() * finite).sum(1), lsm

    if case["op"] == "grad":
        d = torch.zeros(x.shape, dtype=torch.float64, device=x.device)
        none = torch.zeros(T, device=x.device)
        ga, gb = (none if v is None else v for v in (s["ga"], s["gb"]))
        for a in range(0, T, block):
            b = min(T, a + block)
            x64 = x[a:b].double().requires_grad_(True)
            picked, entropy, _ = logp_and_entropy(x64 / tau, a, b)
            (ok[a:b] * (ga[a:b].double() * picked + gb[a:b].double() * entropy)).sum().backward()
            d[a:b] = x64.grad * s["scale"].double()
        return {"dx": d}
    out = {"logp": [], "entropy": [], "saved": [], "top": [], "ids": []}
    for a in range(0, T, block):
        b = min(T, a + block)
        x64 = x[a:b].double()
        picked, entropy, lsm = logp_and_entropy(x64 / tau, a, b)
        largest = x64.max(1).values
        saved = torch.stack([largest, torch.logsumexp((x64 - largest[:, None]) / tau, 1), entropy], 1)
        out["logp"].append(picked * ok[a:b])
        out["entropy"].append(entropy * ok[a:b])
        out["saved"].append(saved * ok[a:b, None])
        if case["k"]:
            ids = torch.sort(x[a:b], dim=1, descending=True, stable=True).indices[:, :case["k"]]
            top = lsm.gather(1, ids)
            ids = ids.masked_fill(torch.isinf(top), -1).masked_fill(~ok[a:b, None], -1)
            out["top"].append(top.masked_fill(~ok[a:b, None], 0.0))
            out["ids"].append(ids.to(s["ids"].dtype))
    return {name: torch.cat(parts) for name, parts in out.items() if parts}
