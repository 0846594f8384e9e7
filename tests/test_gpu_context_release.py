"""Contexts that are dropped in a cycle and collected while another one's update is being captured: the capture ends
well, and its replay computes what the eager calls do."""
import gc

import pytest

torch = pytest.importorskip("torch")

import loss_scaled_adamw_gb300 as tl

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from loss_scaled_adamw_gb300 import _build
    _build.build()


class Step:
    def __init__(self, n=4096):
        g = torch.Generator().manual_seed(1)
        self.master = torch.randn(n, generator=g).cuda()
        self.param = self.master.bfloat16()
        self.state = [torch.zeros(n, device="cuda") for _ in range(3)]
        self.grad = torch.randn(n, generator=g).bfloat16().cuda()
        self.ctx = tl.tl_create([n], [self.param], [self.master], *[[t] for t in self.state], tl.make_config())
        self.hp = tl.tl_adamw_hp(lr=1e-2, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1)

    def update(self):
        tl.logical_update(self.ctx, [[self.grad]], [3], 1.0, self.hp)


def cycle_of(thing):
    cycle = [thing]
    cycle.append(cycle)
    return cycle


def test_collected_inside_a_capture():
    eager, graphed, logits = Step(), Step(), torch.randn(8, 1000, generator=torch.Generator().manual_seed(2)).cuda()
    targets, logp = torch.arange(8, device="cuda"), torch.zeros(8, device="cuda")
    lctx = tl.tl_loss_create(8)
    for step in (eager, graphed):
        step.update()
    tl.tl_token_logprob(lctx, logits, targets, logp)
    want = logp.clone()
    gc.collect()
    held = [cycle_of(Step()), cycle_of(tl.tl_loss_create(64, 4))]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        held.clear()
        gc.collect()
        assert len(tl._dropped) == 2
        graphed.update()
        tl.tl_token_logprob(lctx, logits, targets, logp)
    logp.zero_()
    for _ in range(2):
        graph.replay()
        eager.update()
    torch.cuda.synchronize()
    assert torch.equal(eager.master, graphed.master) and torch.equal(eager.param, graphed.param)
    assert torch.equal(logp, want)
    tl.tl_loss_destroy(tl.tl_loss_create(1))
    assert not tl._dropped
