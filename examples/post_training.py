"""Three post-training objectives on one small model, each trained with the optimizer step, and one of the
caller's own: a policy gradient with an entropy bonus, made of per-token log-probabilities and entropies,
with dropout on the hidden states.

The model is an embedding followed by a linear head over the vocabulary, in fp16 with
dynamic loss scaling; PyTorch does its two matrix products.  Everything from the logits on
is the library's: the objective and the gradient of the logits, multiplied on the device by
the loss scale S, then the accumulation, the overflow check, the norm, the clip, AdamW and
the scaler.  No call reads a device value back until the losses are printed.

    python examples/post_training.py [--steps 60]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import loss_scaled_adamw_gb300 as tl  # noqa: E402

VOCAB, WIDTH, ROWS, TOP = 8192, 128, 256, 16
DROP, BONUS = 0.1, 0.01


class Model:
    """Token t's logits are head @ embedding[t]; the parameters live in an optimizer context."""

    def __init__(self, seed: int):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        shapes = [(VOCAB, WIDTH), (VOCAB, WIDTH)]
        self.masters = [torch.randn(*s, generator=g, device="cuda") * 0.3 for s in shapes]
        self.embedding, self.head = self.params = [w.half() for w in self.masters]
        state = [[torch.zeros_like(w) for w in self.masters] for _ in range(3)]
        cfg = tl.make_config(tl.TL_F16, tl.TL_F16, scaler_enabled=True, init_scale=2.0 ** 12, interval=20)
        self.ctx = tl.tl_create([w.numel() for w in self.masters], self.params, self.masters, *state, cfg)
        self.hp = tl.tl_adamw_hp(lr=5e-3, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.0)

    def logits(self, tokens, key=None):
        """With a key: dropout on the hidden states, whose mask the backward pass draws again."""
        self.hidden, self.key = self.embedding[tokens], key
        if key is not None:
            tl.tl_dropout(self.hidden, self.hidden, DROP, key)
        return self.hidden @ self.head.t()

    def gradients(self, tokens, dlogits):
        """Backward through the two products."""
        g_hidden = dlogits @ self.head
        if self.key is not None:
            tl.tl_dropout(g_hidden, g_hidden, DROP, self.key)
        g_embedding = torch.zeros_like(self.embedding)
        g_embedding.index_add_(0, tokens, g_hidden)
        return [g_embedding, dlogits.t() @ self.hidden]

    def update(self, tokens, dlogits, n: int):
        """Then one logical update of one micro-batch."""
        tl.logical_update(self.ctx, [self.gradients(tokens, dlogits)], [n], max_norm=1.0, hp=self.hp)


def train(name: str, steps: int, lctx):
    """The mean loss of every step (read once at the end)."""
    g = torch.Generator(device="cuda")
    g.manual_seed(7)
    model, result = Model(1), torch.zeros(steps, 4, device="cuda")
    seed = tl.tl_scale_ptr(model.ctx)                    # S, read on the device by every loss
    tokens = torch.randint(0, VOCAB, (ROWS,), generator=g, device="cuda")
    targets = torch.randint(0, VOCAB, (ROWS,), generator=g, device="cuda")
    targets[::8] = -100                                  # positions that carry no loss
    n = ROWS - ROWS // 8
    if name == "distill":                                # a teacher's likeliest entries
        teacher, ids = Model(2).logits(tokens).topk(TOP)
        teacher, ids = teacher.contiguous(), ids.int()
    else:                                                # the starting model is old policy and reference
        ref = torch.zeros(ROWS, device="cuda")
        tl.tl_token_logprob(lctx, model.logits(tokens), targets, ref)
        old, now, advantage = ref.clone(), ref.clone(), torch.ones(ROWS, device="cuda")
        seq = torch.arange(0, ROWS + 1, 16, device="cuda")   # 8 pairs of 16 + 16 rows
    for step in range(steps):
        logits = model.logits(tokens)
        # the gradient replaces the logits: no second matrix of this size
        kw = dict(seed=seed, dlogits=logits)
        if name == "distill":
            tl.tl_distill_loss(lctx, logits, teacher, ids, n, result[step], targets=targets, kd_weight=0.7,
                               ce_weight=0.3, temperature=2.0, **kw)
        elif name == "preference":
            tl.tl_preference_loss(lctx, logits, targets, seq, ROWS // 32, result[step], ref_logp=ref, beta=0.1, **kw)
        else:
            tl.tl_policy_loss(lctx, logits, targets, old, advantage, n, result[step], ref_logp=ref, kl_weight=0.01,
                              logp=now, **kw)
            if step % 4 == 3:                            # four updates per sample
                old.copy_(now)
        model.update(tokens, logits, n)
    return result[:, 0].tolist(), tl.tl_read_status(model.ctx)


class Bonus:
    """The mean over n tokens of -advantage * log-probability - BONUS * entropy: forward by tl_token_stats,
    gradient of the logits by tl_token_grad from the derivatives for each token."""

    def __init__(self, lctx, targets, advantage, n: int, seed):
        self.lctx, self.targets, self.seed = lctx, targets, seed
        self.valid = (targets >= 0).float()
        self.g_logp, self.g_entropy = -advantage * self.valid / n, -BONUS * self.valid / n
        rows = targets.shape[0]
        self.logp, self.entropy = torch.zeros(rows, device="cuda"), torch.zeros(rows, device="cuda")
        self.saved = torch.zeros(rows, 3, device="cuda")

    def loss(self, logits):
        tl.tl_token_stats(self.lctx, logits, self.targets, logp=self.logp, entropy=self.entropy, saved=self.saved)
        return (self.g_logp * self.logp + self.g_entropy * self.entropy).sum()

    def gradient(self, logits):
        """In the place of the logits."""
        tl.tl_token_grad(self.lctx, logits, self.saved, logits, self.targets, self.g_logp, self.g_entropy, seed=self.seed)


def train_bonus(steps: int, lctx):
    g = torch.Generator(device="cuda")
    g.manual_seed(7)
    model, losses = Model(1), torch.zeros(steps, device="cuda")
    tokens = torch.randint(0, VOCAB, (ROWS,), generator=g, device="cuda")
    targets = torch.randint(0, VOCAB, (ROWS,), generator=g, device="cuda")
    targets[::8] = -100
    n = ROWS - ROWS // 8
    bonus = Bonus(lctx, targets, torch.ones(ROWS, device="cuda"), n, tl.tl_scale_ptr(model.ctx))
    key = torch.tensor([7, 0], dtype=torch.int64, device="cuda")      # seed, ticket
    for step in range(steps):
        logits = model.logits(tokens, key)
        losses[step] = bonus.loss(logits)
        bonus.gradient(logits)
        model.update(tokens, logits, n)
        key[1:].add_(1)                                  # another mask for the next micro-batch
    return losses.tolist(), tl.tl_read_status(model.ctx)


def main():
    parser = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    parser.add_argument("--steps", type=int, default=60)
    steps = parser.parse_args().steps
    lctx = tl.tl_loss_create(max_rows=ROWS, max_pairs=ROWS // 32)
    for name in ("distill", "preference", "policy"):
        losses, status = train(name, steps, lctx)
        report(name, losses, status)
    report("bonus", *train_bonus(steps, lctx))


def report(name, losses, status):
    print(f"{name:10s} loss {losses[0]:.4f} -> {losses[-1]:.4f}   steps committed {status.t}, S = {status.S:g}")


if __name__ == "__main__":
    main()
