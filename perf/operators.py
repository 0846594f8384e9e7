"""The objectives over vocabulary logits as measured work: cases, inputs, plain forms, exact values.

Each case is one call of tl_token_logprob, tl_policy_loss, tl_preference_loss or
tl_distill_loss.  `run` computes it in its plain form (elementary torch operations in
fp32, rounded once at the end) or, with `own` set, through the library.  `exact` gives
the same outputs from the definition in fp64, the gradients by automatic
differentiation of the loss.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
IGNORED = -100

# 4,096 rows are the 8 x 512 positions of a micro-batch, and 128,256 and 8,192 entries the
# vocabularies of the llama_1b and llama_10m workloads; 50,001 and 32,003 are odd
# vocabularies, whose rows start at every element phase.
ROWS, VOCAB, VOCAB_SMALL, VOCAB_ODD = 4096, 128256, 8192, 50001
MOST_BYTES = 2 * ROWS * VOCAB * 2            # a pass over the largest case: logits in, gradients out


def listed():
    return [
        # scoring the one token just sampled with the large vocabulary: latency
        _case("logprob_one_token", "logprob", 1, VOCAB, "bf16"),
        # old log-probabilities of a few thousand rows from fp32 logits, odd vocabulary, sampling temperature
        _case("logprob_odd_f32", "logprob", 1500, 32003, "f32", tau=0.7, masked=0.1),
        # the reference model's log-probabilities of a whole micro-batch
        _case("logprob_llama_1b", "logprob", ROWS, VOCAB, "bf16", masked=0.125),
        # a policy update on a few short answers of the small model
        _case("policy_small", "policy", 64, VOCAB_SMALL, "f16", masked=0.125, ref=True),
        # no KL term, odd vocabulary: rows at every alignment
        _case("policy_odd", "policy", 777, VOCAB_ODD, "bf16", masked=0.3),
        # a whole micro-batch of the large model with the KL term
        _case("policy_llama_1b", "policy", ROWS, VOCAB, "bf16", masked=0.125, ref=True),
        # two pairs of short answers, fp32 logits: latency of the two dependent passes
        _case("preference_small", "preference", 96, VOCAB_SMALL, "f32", pairs=2, masked=0.25, ref=True),
        # ragged pairs without a reference model, label smoothing, fp16 with a loss scale
        _case("preference_odd", "preference", 1111, 32003, "f16", pairs=5, masked=0.4, smooth=0.1),
        # eight pairs of long sequences of the large model, a quarter of the rows prompt
        _case("preference_llama_1b", "preference", ROWS, VOCAB, "bf16", pairs=8, masked=0.25, ref=True),
        # a small student, few teacher entries, soft targets alone
        _case("distill_small", "distill", 32, VOCAB_SMALL, "f32", k=8, tau=1.0),
        # odd vocabulary, 64-bit ids, odd number of teacher entries, one temperature for both terms
        _case("distill_odd", "distill", 513, VOCAB_ODD, "f16", k=101, tau=1.0, ce=0.5, masked=0.1, wide_ids=True),
        # a whole micro-batch of the large model at temperature 2 beside the hard targets
        _case("distill_llama_1b", "distill", ROWS, VOCAB, "bf16", k=64, tau=2.0, ce=0.25, masked=0.125),
    ]


def _case(name, op, rows, vocab, dtype, tau=1.0, masked=0.0, ref=False, pairs=0, smooth=0.0, k=0, ce=0.0,
          wide_ids=False):
    return {"name": name, "op": op, "rows": rows, "vocab": vocab, "dtype": dtype, "tau": tau, "masked": masked,
            "ref": ref, "pairs": pairs, "smooth": smooth, "k": k, "ce": ce, "wide_ids": wide_ids}


def draw(rng):
    log = lambda lo, hi: int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))  # noqa: E731
    op = rng.choice(["logprob", "policy", "preference", "distill"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    vocab = log(500, VOCAB)
    if rng.random() < 0.5:
        vocab = max(512, vocab // 64 * 64)          # half of them padded to a round size, the rest as they come
    size = 4 if dtype == "f32" else 2
    rows = min(log(1, 4 * ROWS), max(1, MOST_BYTES // (2 * size * vocab)))
    c = _case("", op, rows, vocab, dtype, tau=rng.choice([1.0, 1.0, 0.7, 2.0]), masked=rng.choice([0.0, 0.125, 0.4]))
    del c["name"]
    if op == "policy":
        c["ref"] = rng.random() < 0.7
    if op == "preference":
        c["rows"] = max(4, c["rows"])
        c["pairs"] = max(1, min(log(1, 64), c["rows"] // 4))
        c["ref"] = rng.random() < 0.7
        c["smooth"] = rng.choice([0.0, 0.0, 0.1])
    if op == "distill":
        c["k"] = min(log(1, 256), vocab)
        c["ce"] = rng.choice([0.0, 0.25, 0.5])
        c["wide_ids"] = rng.random() < 0.3
    return c


def _lengths(case):
    """The lengths of the 2 * pairs sequences of a preference case (the same for every seed)."""
    n = 2 * case["pairs"]
    r = random.Random(case["rows"] * 1009 + n)
    cuts = sorted(r.sample(range(1, case["rows"]), n - 1))
    return [b - a for a, b in zip([0] + cuts, cuts + [case["rows"]])]


def _mask(case):
    """The ignored rows (the same for every seed): the start of each sequence in a preference case, whose prompt
    carries no loss; the padded end of each 512-row sequence otherwise."""
    ignored = [False] * case["rows"]
    at = 0
    if case["op"] == "preference":
        for n in _lengths(case):
            for i in range(at, at + int(n * case["masked"])):
                ignored[i] = True
            at += n
    else:
        while at < case["rows"]:
            n = min(512, case["rows"] - at)
            for i in range(at + n - int(n * case["masked"]), at + n):
                ignored[i] = True
            at += n
    return ignored


def _log_softmax(x, tau):
    return torch.log_softmax(x.float() / tau, -1)


def prepare(case, seed):
    T, V, dev = case["rows"], case["vocab"], "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    def uniform(*shape):
        return torch.rand(*shape, generator=g, device=dev)

    s = {"case": dict(case)}
    # logits of a language model: a broad spread, the label among the likely entries
    target = torch.randint(0, V, (T,), generator=g, device=dev)
    x = normal(T, V) * 2.5
    x[torch.arange(T, device=dev), target] += 2 + 12 * uniform(T)
    x = x.to(DTYPES[case["dtype"]])
    ignored = torch.tensor(_mask(case), device=dev)
    s["x"], s["target"] = x, torch.where(ignored, IGNORED, target)
    valid = int(T - sum(_mask(case)))
    s["n"] = max(1, case["pairs"] if case["op"] == "preference" else valid)
    s["scale"] = torch.full((1,), 2.0 ** 14 if case["dtype"] == "f16" else 1.0, device=dev)
    if case["op"] != "logprob":
        s["dx"] = torch.empty_like(x)
        s["result"] = torch.zeros(4, device=dev)
    s["row"] = torch.zeros(T, device=dev)
    s["logp"] = torch.zeros(T, device=dev)
    if case["op"] in ("policy", "preference"):
        lp = torch.empty(T, device=dev)
        for a in range(0, T, 1024):
            lp[a:a + 1024] = _log_softmax(x[a:a + 1024], case["tau"]).gather(1, target[a:a + 1024, None])[:, 0]
        s["ref"] = lp + 0.3 * normal(T) if case["ref"] else None
    if case["op"] == "policy":
        # the policy has moved a little since the sample was drawn: most ratios within the clip
        # range, some beyond it, none so near its edge that rounding would decide
        d = 0.15 * normal(T)
        for edge in (math.log(0.8), math.log(1.2)):
            d = torch.where((d - edge).abs() < 2e-3, d + 5e-3, d)
        s["old"] = lp - d
        s["adv"] = normal(T)
    if case["op"] == "preference":
        n = torch.tensor(_lengths(case), dtype=torch.int64)
        s["seq"] = torch.cat([torch.zeros(1, dtype=torch.int64), torch.cumsum(n, 0)]).to(dev)
        s["pair"] = torch.zeros(case["pairs"], device=dev)
        s["reward"] = torch.zeros(2 * case["pairs"], device=dev)
    if case["op"] == "distill":
        # the teacher's likeliest entries, the label mostly among them, ids in no order
        key = uniform(T, V)
        key[torch.arange(T, device=dev), target] -= (uniform(T) < 0.9).float()
        ids = key.topk(case["k"], largest=False).indices
        ids = ids.gather(1, uniform(T, case["k"]).argsort(1))
        s["t_ids"] = ids.contiguous() if case["wide_ids"] else ids.int()
        s["t_logits"] = (normal(T, case["k"]) * 2 + 6 * (ids == target[:, None])).to(
            torch.float32 if case["dtype"] == "f32" else torch.bfloat16)
        del key
    return s


def _softmax_parts(x32):
    """Per row: x - max, exp of it, the sum of those."""
    z = x32 - x32.amax(1, keepdim=True)
    e = z.exp()
    return z, e, e.sum(1)


def _plain(s):
    c = s["case"]
    tau, valid = c["tau"], s["target"] >= 0
    y = s["target"].clamp(min=0)[:, None]
    x32 = s["x"].float()
    z, e, total = _softmax_parts(x32 / tau)
    lp = torch.where(valid, z.gather(1, y)[:, 0] - total.log(), 0.0)
    if c["op"] == "logprob":
        return {"logp": lp}
    step = s["scale"] / s["n"]

    def mean(v):
        return torch.where(valid, v, 0.0).sum() / s["n"]

    def gradient(g):
        """g: dL/dlogp of each row."""
        w = torch.where(valid, g * step / tau, 0.0)[:, None]
        d = e * (-w / total[:, None])
        d.scatter_add_(1, y, w)
        return d.masked_fill_(~valid[:, None], 0.0).to(s["x"].dtype)

    if c["op"] == "policy":
        r = (lp - s["old"]).exp()
        free, held = r * s["adv"], r.clamp(0.8, 1.2) * s["adv"]
        surrogate = -torch.minimum(free, held)
        g = torch.where(free <= held, -free, 0.0)
        kl = torch.zeros_like(lp)
        if s["ref"] is not None:
            b = s["ref"] - lp
            kl = b.exp() - b - 1
            g = g + KL * (1 - b.exp())
        row = torch.where(valid, surrogate + KL * kl, 0.0)
        result = torch.stack([mean(row), mean(surrogate), mean(kl), valid.sum().float()])
        return {"dx": gradient(g), "logp": lp, "row": row, "result": result}

    if c["op"] == "preference":
        ratio = lp if s["ref"] is None else torch.where(valid, lp - s["ref"], 0.0)
        at = torch.cat([torch.zeros(1, device=lp.device), ratio]).double().cumsum(0)[s["seq"]]
        reward = (BETA * (at[1:] - at[:-1])).float()
        h = reward[0::2] - reward[1::2]
        up, down = 1 / (1 + (-h).exp()), 1 / (1 + h.exp())
        pair = -(1 - c["smooth"]) * up.log() - c["smooth"] * down.log()
        dh = -BETA * ((1 - c["smooth"]) * down - c["smooth"] * up)
        per_seq = torch.stack([dh, -dh], 1).reshape(-1)
        g = per_seq.repeat_interleave(s["seq"][1:] - s["seq"][:-1])
        n = s["n"]
        result = torch.stack([pair.sum() / n, h.sum() / n, (h > 0).sum() / n, (h == h).sum().float()])
        return {"dx": gradient(g), "logp": lp, "pair": pair, "reward": reward, "result": result}

    tz, te, tt = _softmax_parts(s["t_logits"].float() / tau)
    p = te / tt[:, None]
    ids = s["t_ids"].long()
    log_q = z.gather(1, ids) - total.log()[:, None]
    kd = tau * tau * (p * (tz - tt.log()[:, None] - log_q)).sum(1)
    w = step * KD * tau
    d = (e * (w / total[:, None])).scatter_add_(1, ids, -w * p)
    row, ce = KD * kd, torch.zeros_like(kd)
    if c["ce"]:
        z1, e1, total1 = _softmax_parts(x32)
        ce = total1.log() - z1.gather(1, y)[:, 0]
        row = row + c["ce"] * ce
        v = step * c["ce"]
        d += e1 * (v / total1[:, None])
        d.scatter_add_(1, y, -v.expand(y.shape[0])[:, None])
    row = torch.where(valid, row, 0.0)
    result = torch.stack([mean(row), mean(kd), mean(ce), valid.sum().float()])
    return {"dx": d.masked_fill_(~valid[:, None], 0.0).to(s["x"].dtype), "row": row, "result": result}


KL, BETA, KD = 0.05, 0.1, 0.75


def run(state):
    return _own(state) if own else _plain(state)


_context = None


def _own(s):
    import loss_scaled_adamw_gb300 as tl
    global _context
    if _context is None:      # one context for a process, as a trainer keeps it
        _context = tl.tl_loss_create(max_rows=4 * ROWS, max_pairs=64)
    c, x = s["case"], s["x"]
    if c["op"] == "logprob":
        tl.tl_token_logprob(_context, x, s["target"], s["logp"], temperature=c["tau"])
        return {"logp": s["logp"]}
    if c["op"] == "policy":
        tl.tl_policy_loss(_context, x, s["target"], s["old"], s["adv"], s["n"], s["result"], ref_logp=s["ref"],
                          clip_low=0.2, clip_high=0.2, kl_weight=KL if c["ref"] else 0.0, temperature=c["tau"],
                          seed=s["scale"], dlogits=s["dx"], logp=s["logp"], row_loss=s["row"])
        return {"dx": s["dx"], "logp": s["logp"], "row": s["row"], "result": s["result"]}
    if c["op"] == "preference":
        tl.tl_preference_loss(_context, x, s["target"], s["seq"], s["n"], s["result"], ref_logp=s["ref"], beta=BETA,
                              label_smoothing=c["smooth"], temperature=c["tau"], seed=s["scale"], dlogits=s["dx"],
                              logp=s["logp"], pair_loss=s["pair"], reward=s["reward"])
        return {"dx": s["dx"], "logp": s["logp"], "pair": s["pair"], "reward": s["reward"], "result": s["result"]}
    tl.tl_distill_loss(_context, x, s["t_logits"], s["t_ids"], s["n"], s["result"], targets=s["target"],
                       kd_weight=KD, ce_weight=c["ce"], temperature=c["tau"], seed=s["scale"], dlogits=s["dx"],
                       row_loss=s["row"])
    return {"dx": s["dx"], "row": s["row"], "result": s["result"]}


def work(case):
    """Logits of the rows that carry loss read once, every gradient row written once, the row
    inputs and outputs; about ten operations per logit and direction."""
    T, V = case["rows"], case["vocab"]
    size = 4 if case["dtype"] == "f32" else 2
    valid = T - sum(_mask(case))
    read = valid * V * size + 8 * T
    if case["op"] == "logprob":
        return {"bytes": read + 4 * T, "flops": 5 * valid * V}
    more = {"policy": (8 + 4 * case["ref"]) * T + 8 * T, "preference": (4 + 4 * case["ref"]) * T,
            "distill": valid * case["k"] * ((8 if case["wide_ids"] else 4) + (4 if size == 4 else 2)) + 4 * T}[case["op"]]
    return {"bytes": read + T * V * size + more, "flops": (18 if case["ce"] and case["tau"] != 1 else 10) * valid * V}


def exact(case, seed):
    """The definition in fp64, blocks of rows at a time; gradients by automatic differentiation."""
    s = prepare(case, seed)
    T, tau = case["rows"], case["tau"]
    x, tgt = s["x"], s["target"]
    block = max(1, (1 << 25) // case["vocab"])
    spans = [(a, min(T, a + block)) for a in range(0, T, block)]

    def logprob(x64, a, b):
        lsm = torch.nn.functional.log_softmax(x64 / tau, dim=1)
        return lsm[torch.arange(b - a, device=x.device), tgt[a:b].clamp(min=0)] * (tgt[a:b] >= 0)

    def gradients(loss_of_block):
        d = torch.empty(x.shape, dtype=torch.float64, device=x.device)
        for a, b in spans:
            x64 = x[a:b].double().requires_grad_(True)
            loss_of_block(x64, a, b).backward()
            d[a:b] = x64.grad * (s["scale"].double() / s["n"])
        return d

    ok = (tgt >= 0)
    if case["op"] in ("logprob", "policy", "preference"):
        lp = torch.cat([logprob(x[a:b].double(), a, b) for a, b in spans])
        if case["op"] == "logprob":
            return {"logp": lp}
        ref = None if s["ref"] is None else s["ref"].double()
        leaf = lp.clone().requires_grad_(True)
    n = s["n"]
    if case["op"] == "policy":
        ratio = torch.exp(leaf - s["old"].double())
        adv = s["adv"].double()
        sur = -torch.min(ratio * adv, torch.clip(ratio, 0.8, 1.2) * adv) * ok
        kl = torch.zeros_like(sur) if ref is None else (torch.expm1(ref - leaf) - (ref - leaf)) * ok
        row = sur + KL * kl
        row.sum().backward()
        out = [row.detach().sum() / n, sur.detach().sum() / n, kl.detach().sum() / n, ok.sum().double()]
        g = leaf.grad
        return {"dx": gradients(lambda x64, a, b: (logprob(x64, a, b) * g[a:b]).sum()), "logp": lp,
                "row": row.detach(), "result": torch.stack(out)}
    if case["op"] == "preference":
        rel = leaf if ref is None else (leaf - ref) * ok
        reward = BETA * torch.stack([part.sum() for part in rel.split(_lengths(case))])
        margin = reward[0::2] - reward[1::2]
        sig = torch.nn.functional.logsigmoid
        pair = -(1 - case["smooth"]) * sig(margin) - case["smooth"] * sig(-margin)
        pair.sum().backward()
        out = [pair.detach().sum() / n, margin.detach().sum() / n, (margin > 0).double().sum() / n,
               torch.full((), float(case["pairs"]), dtype=torch.float64, device=x.device)]
        g = leaf.grad
        return {"dx": gradients(lambda x64, a, b: (logprob(x64, a, b) * g[a:b]).sum()), "logp": lp,
                "pair": pair.detach(), "reward": reward.detach(), "result": torch.stack(out)}

    rows, kds, ces = [], [], []

    def block_loss(x64, a, b):
        p = torch.softmax(s["t_logits"][a:b].double() / tau, 1)
        lsm = torch.nn.functional.log_softmax(x64 / tau, dim=1).gather(1, s["t_ids"][a:b].long())
        kd = tau ** 2 * (p * (p.log() - lsm)).sum(1) * ok[a:b]
        ce = torch.zeros_like(kd)
        if case["ce"]:
            pick = torch.nn.functional.log_softmax(x64, dim=1)
            ce = -pick.gather(1, tgt[a:b].clamp(min=0)[:, None])[:, 0] * ok[a:b]
        row = KD * kd + case["ce"] * ce
        rows.append(row.detach()), kds.append(kd.detach()), ces.append(ce.detach())
        return row.sum()

    d = gradients(block_loss)
    row = torch.cat(rows)
    return {"dx": d, "row": row, "result": torch.stack([row.sum() / n, torch.cat(kds).sum() / n, torch.cat(ces).sum() / n,
                                                        ok.sum().double()])}
