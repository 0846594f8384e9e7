"""Row statistics, their gradient and dropout used together: a teacher's entries on their way into distillation, and
the example's objective of its own (dropout, log-probabilities and entropies, their gradient, dropout backwards)."""
import importlib.util
import math
import os

import pytest

torch = pytest.importorskip("torch")

import loss_reference as L
import loss_scaled_adamw_gb300 as tl
import token_reference as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lctx():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from loss_scaled_adamw_gb300 import _build
    _build.build()
    return tl.tl_loss_create(1024, 8)


@pytest.fixture(scope="module")
def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "post_training.py")
    spec = importlib.util.spec_from_file_location("post_training", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("T,V,k", [(37, 1003, 20), (5, 40000, 64), (300, 9000, 7)])
def test_teacher_entries_into_distillation(lctx, T, V, k):
    """The entries' log-probabilities stand for the teacher's logits: the loss is that of its k largest logits.  KD is
    a mean of differences of log-probabilities: off by their errors (4e-5 and a few eps), times tau^2."""
    g = torch.Generator().manual_seed(V)
    teacher, student = torch.randn(T, V, generator=g) * 3, (torch.randn(T, V, generator=g) * 2).bfloat16()
    y = torch.randint(0, V, (T,), generator=g)
    y[1] = -1
    n, tau = T - 1, 2.0
    ids, top = torch.zeros(T, k, dtype=torch.int32, device="cuda"), torch.zeros(T, k, device="cuda")
    tl.tl_token_stats(lctx, teacher.cuda(), top_ids=ids, top_logp=top)
    result, rows = torch.zeros(4, device="cuda"), torch.zeros(T, device="cuda")
    d = torch.zeros_like(student, device="cuda")
    tl.tl_distill_loss(lctx, student.cuda(), top, ids, n, result, targets=y.cuda(), kd_weight=0.7, ce_weight=0.3,
                       temperature=tau, dlogits=d, row_loss=rows)
    want_ids = torch.sort(teacher, dim=1, descending=True, stable=True).indices[:, :k]
    assert torch.equal(ids.cpu().long(), want_ids)
    want = L.distill(student, teacher.gather(1, want_ids), want_ids, n, y, 0.7, 0.3, tau, 1.0)
    assert (rows.cpu().double() - want["loss"]).abs().max() < 4e-4
    assert (d.cpu().double() - want["dx"]).abs().max() < 2.0 ** -8 * want["dx"].abs().max() + 1e-6


def test_example_objective_of_its_own(lctx, example):
    losses, status = example.train_bonus(12, lctx)
    assert all(math.isfinite(v) for v in losses) and status.t >= 10 and status.found_inf == 0


def test_example_gradients(lctx, example):
    """The gradients of embedding and head against automatic differentiation in fp64, with the mask drawn apart.  The
    example's products round logits (of at most 16) and gradients to fp16: an exponent is off by 16 * 2^-12, so a
    probability by 0.4 %, and each later rounding adds 2^-11 of a term: 1 % of the gradients' norm bounds it."""
    model, n, S = example.Model(1), 224, 4096.0
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    tokens = torch.randint(0, example.VOCAB, (256,), generator=g, device="cuda")
    targets = torch.randint(0, example.VOCAB, (256,), generator=g, device="cuda")
    targets[::8] = -100
    advantage = torch.randn(256, generator=g, device="cuda")
    key = torch.tensor([11, 4], dtype=torch.int64, device="cuda")
    bonus = example.Bonus(lctx, targets, advantage, n, tl.tl_scale_ptr(model.ctx))
    logits = model.logits(tokens, key)
    assert logits.abs().max() < 16
    loss = bonus.loss(logits)
    bonus.gradient(logits)
    got = model.gradients(tokens, logits)

    w = [p.double().requires_grad_(True) for p in model.params]
    P = round(example.DROP * 65536)
    keep = torch.from_numpy(R.numbers(0, 256 * example.WIDTH, 11, 4, 0) >= P).view(256, example.WIDTH).cuda()
    x = w[0][tokens] * keep / (1 - P / 65536) @ w[1].t()
    lsm = torch.log_softmax(x, 1)
    logp = lsm.gather(1, targets.clamp(min=0)[:, None])[:, 0]
    entropy = -(lsm.exp() * lsm).sum(1)
    want = ((-advantage * logp - example.BONUS * entropy) * (targets >= 0)).sum() / n
    want.backward()
    want = float(want.detach())
    assert abs(float(loss) - want) < 1e-2 * abs(want) + 1e-2
    for a, b in zip(got, w):
        assert (a.double() / S - b.grad).norm() < 1e-2 * b.grad.norm()
