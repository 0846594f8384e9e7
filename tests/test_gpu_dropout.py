"""Dropout on the GPU against its statement in fp64 (token_reference.py).

An element is one multiply-add in fp32 and one rounding to the type: the scale rounds by eps = 2^-24 of itself, the
multiply-add once more, so y is off by 2 eps |x / (1 - p)| + eps |y| and half a step of the type.  Which elements are
kept has to be equal.
"""
import pytest

torch = pytest.importorskip("torch")

import loss_scaled_adamw_gb300 as tl
import token_reference as R

pytestmark = pytest.mark.gpu

EPS = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from loss_scaled_adamw_gb300 import _build
    _build.build()


def matrix(rows, cols, dtype, pad, lead, seed):
    g = torch.Generator().manual_seed(seed)
    buf = torch.randn(lead + rows * (cols + pad) + 16, generator=g).to(DT[dtype]).cuda()
    return buf[lead:lead + rows * (cols + pad)].view(rows, cols + pad)[:, :cols], buf


def check(got, x, p, seed, ticket, site, res=None):
    x, got, res = x.cpu(), got.cpu(), None if res is None else res.cpu()
    want = R.dropout(x, p, seed, ticket, site, res)
    scale = 1 / max(1 - p, 1e-5)
    tol = 2 * EPS * x.double().abs() * scale + want.abs() * (EPS + torch.finfo(x.dtype).eps / 2 * 1.01) + \
        {torch.float16: 2.0 ** -25, torch.bfloat16: 1e-38, torch.float32: 1e-38}[x.dtype]
    off = (got.double() - want).abs()
    assert (off <= tol).all(), (off.max(), got.flatten()[:8], want.flatten()[:8])
    if res is None:
        keep = torch.from_numpy(R.numbers(0, x.numel(), seed, ticket, site) >= round(p * 65536)).view(x.shape)
        assert torch.equal((got != 0) & (x != 0), keep & (x != 0))


CASES = [(1, 1, 0, 0), (1, 7, 0, 0), (1, 8, 0, 0), (1, 2048, 0, 0), (1, 4099, 0, 0), (1, 4099, 0, 3), (1, 20001, 0, 5), (3, 5, 0, 0), (3, 5, 2, 1),
         (17, 64, 0, 0), (17, 64, 8, 0), (17, 64, 8, 1), (17, 64, 3, 0), (33, 1153, 6, 3), (9, 8192, 64, 8), (40, 288, 0, 0),
         (1000, 129, 0, 0), (300, 2048, 0, 0), (70, 16392, 16, 0), (23, 8192, 7, 3), (11, 4097, 6, 5), (40, 700, 3, 0), (9, 1031, 2, 7), (13, 513, 0, 0), (6, 2049, 1, 6), (500, 3, 1, 0), (257, 1, 1, 0), (5, 2051, 5, 4)]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,cols,pad,lead", CASES)
def test_sizes_strides_and_alignment(rows, cols, pad, lead, dtype):
    seed, ticket, site = 0x1234567890 + rows, 3 + cols, 5
    key = torch.tensor([seed, ticket], dtype=torch.int64, device="cuda")
    x, _ = matrix(rows, cols, dtype, pad, lead, 1)
    res, _ = matrix(rows, cols, dtype, pad, lead, 2)
    for p, r in ((0.1, None), (0.5, res), (0.75, None), (0.1, res)):
        y, buf = matrix(rows, cols, dtype, pad, lead, 3)
        before = buf.clone()
        tl.tl_dropout(x, y, p, key, site=site, residual=r)
        check(y, x, p, seed, ticket, site, r)
        after = buf.clone()
        torch.as_strided(after, y.shape, y.stride(), y.storage_offset()).copy_(
            torch.as_strided(before, y.shape, y.stride(), y.storage_offset()))
        assert torch.equal(after, before)                     # nothing between or behind the rows


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_operands_of_different_strides_and_phases(dtype):
    seed, ticket, site = 77, 1, 0
    key = torch.tensor([seed, ticket], dtype=torch.int64, device="cuda")
    for (px, lx), (pr, lr), (py, ly) in (((0, 0), (8, 0), (0, 0)), ((0, 0), (0, 1), (0, 0)), ((8, 8), (16, 0), (24, 0)),
                                         ((1, 0), (2, 3), (0, 0)), ((4, 4), (12, 4), (8, 4))):
        x, r, y = matrix(21, 96, dtype, px, lx, 1)[0], matrix(21, 96, dtype, pr, lr, 2)[0], matrix(21, 96, dtype, py, ly, 3)[0]
        tl.tl_dropout(x, y, 0.3, key, residual=r)
        check(y, x, 0.3, seed, ticket, site, r)


def test_mask_does_not_depend_on_type_shape_or_strides():
    key = torch.tensor([5, 9], dtype=torch.int64, device="cuda")
    ones, masks = torch.ones(24 * 40), []
    for t in (ones.cuda(), ones.bfloat16().cuda().view(24, 40), ones.half().cuda().view(4, 6, 40),
              matrix(24, 40, "bf16", 5, 1, 1)[0].fill_(1.0), matrix(24, 40, "f32", 8, 0, 1)[0].fill_(1.0)):
        y = torch.empty_like(t) if t.is_contiguous() else matrix(24, 40, "bf16" if t.dtype == torch.bfloat16 else "f32", 3, 2, 1)[0]
        tl.tl_dropout(t, y, 0.4, key, site=2)
        masks.append((y != 0).flatten().cpu())
    assert all(torch.equal(m, masks[0]) for m in masks)


def test_key_site_and_ticket_change_the_mask():
    x, y = torch.ones(4096, device="cuda"), torch.empty(4096, device="cuda")
    seen = []
    for seed, ticket, site in ((1, 0, 0), (2, 0, 0), (1 << 40, 0, 0), (-1, 0, 0), (1, 1, 0), (1, 1 << 33, 0), (1, 0, 1), (1, 0, 2 ** 32 - 1)):
        tl.tl_dropout(x, y, 0.5, torch.tensor([seed, ticket], device="cuda"), site=site)
        check(y, x, 0.5, seed, ticket, site)
        seen.append(y.clone())
    assert all(not torch.equal(a, b) for i, a in enumerate(seen) for b in seen[:i])


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("cols,pad", [(512, 0), (513, 0), (129, 2)])
def test_no_and_all_dropped(cols, pad, dtype):
    key = torch.tensor([1, 2], dtype=torch.int64, device="cuda")
    x, res = matrix(6, cols, dtype, pad, 0, 1)[0], matrix(6, cols, dtype, pad, 0, 2)[0]
    y = torch.empty_like(x)
    tl.tl_dropout(x, y, 0.0, key)
    assert torch.equal(y, x)
    tl.tl_dropout(x, y, 2.0 ** -18, key)                 # rounds to 0
    assert torch.equal(y, x)
    x.fill_(NAN)
    tl.tl_dropout(x, y, 1.0, key)
    assert (y == 0).all()
    tl.tl_dropout(x, y, 1.0, key, residual=res)
    assert torch.equal(y, res)
    tl.tl_dropout(x, y, 0.5, key)                        # dropped elements are 0 whatever they hold
    keep = torch.from_numpy(R.numbers(0, x.numel(), 1, 2, 0) >= 32768).view(x.shape)
    assert torch.equal(torch.isnan(y).cpu(), keep) and (y.cpu()[~keep] == 0).all()
    x.fill_(-INF)
    tl.tl_dropout(x, y, 0.5, key)
    assert torch.equal(torch.isinf(y).cpu(), keep)


@pytest.mark.parametrize("pad", [0, 8, 3])
def test_in_place(pad):
    key = torch.tensor([3, 4], dtype=torch.int64, device="cuda")
    x, r = matrix(30, 200, "bf16", pad, 0, 1)[0], matrix(30, 200, "bf16", pad, 0, 2)[0]
    want, both = torch.empty_like(x), torch.empty_like(x)
    tl.tl_dropout(x, want, 0.2, key)
    tl.tl_dropout(x, both, 0.2, key, residual=r)
    into_res = matrix(30, 200, "bf16", pad, 0, 2)[0]
    tl.tl_dropout(x, into_res, 0.2, key, residual=into_res)
    assert torch.equal(into_res, both)
    tl.tl_dropout(x, x, 0.2, key, residual=r)
    assert torch.equal(x, both)


def test_gradient_is_the_same_call():
    """<dropout(x), g> is linear in x: differences of one step are the gradient of every element."""
    key = torch.tensor([11, 5], dtype=torch.int64, device="cuda")
    x, g = torch.zeros(500, device="cuda"), torch.randn(500, generator=torch.Generator().manual_seed(1)).cuda()
    d, y = torch.empty_like(x), torch.empty_like(x)
    tl.tl_dropout(g, d, 0.25, key, site=4)
    for i in range(0, 500, 7):
        e = x.clone()
        e[i] = 1.0
        tl.tl_dropout(e, y, 0.25, key, site=4)
        assert float((y * g).sum()) == float(d[i])


def test_share_kept():
    x, y = torch.ones(1 << 20, device="cuda"), torch.empty(1 << 20, device="cuda")
    for p in (0.1, 0.5, 0.9):
        tl.tl_dropout(x, y, p, torch.tensor([123, 456], device="cuda"))
        kept = float((y != 0).float().mean())
        assert abs(kept - (1 - p)) < 5 * (p * (1 - p)) ** 0.5 / 1024 + 2.0 ** -16     # five standard deviations


def test_refusals():
    key = torch.tensor([1, 2], dtype=torch.int64, device="cuda")
    x, y = torch.zeros(8, 32, device="cuda"), torch.zeros(8, 32, device="cuda")
    for kw in (dict(p=-0.1), dict(p=1.1), dict(p=NAN)):
        with pytest.raises(tl.TLError):
            tl.tl_dropout(x, y, key=key, **kw)
    flat = torch.zeros(300, device="cuda")
    with pytest.raises(tl.TLError):
        tl.tl_dropout(flat[:256], flat[8:264], 0.1, key)
    with pytest.raises(tl.TLError):
        tl.tl_dropout(x, y, 0.1, y.view(torch.int64)[0, :2])
    for bad in (dict(x=x.cpu()), dict(y=y.cpu()), dict(y=y.half()), dict(y=y[:, :16]), dict(key=key.int()), dict(key=key[:1]),
                dict(key=None), dict(site=-1), dict(site=2 ** 32), dict(x=x.double(), y=y.double()), dict(residual=x.t()),
                dict(x=x.t(), y=y.t()), dict(x=None)):
        a = dict(x=x, y=y, p=0.1, key=key)
        a.update(bad)
        with pytest.raises((ValueError, tl.TLError)):
            tl.tl_dropout(**a)
    tl.tl_dropout(x[:0], y[:0], 0.1, key)


def test_captured_with_a_ticket_that_advances():
    key = torch.tensor([21, 0], dtype=torch.int64, device="cuda")
    x = torch.randn(64, 256, generator=torch.Generator().manual_seed(3)).bfloat16().cuda()
    y, d = torch.empty_like(x), torch.empty_like(x)

    def step():
        key[1:].add_(1)
        tl.tl_dropout(x, y, 0.1, key, site=1, residual=x)
        tl.tl_dropout(x, d, 0.1, key, site=1)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    key[1] = 100
    for ticket in (101, 102, 103):
        graph.replay()
        check(y, x, 0.1, 21, ticket, 1, x)
        check(d, x, 0.1, 21, ticket, 1)


def test_far_elements():
    """Element offsets beyond 2^31 and 2^32."""
    free, _ = torch.cuda.mem_get_info()
    n = (1 << 32) + 4099
    if free < 2 * 2 * n + (1 << 30):
        pytest.skip("not enough memory")
    key = torch.tensor([9, 1], dtype=torch.int64, device="cuda")
    x = torch.ones(n, dtype=torch.bfloat16, device="cuda")
    y = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    tl.tl_dropout(x, y, 0.5, key)
    for first in (0, (1 << 31) - 40, (1 << 32) - 40, n - 5000):
        keep = torch.from_numpy(R.numbers(first, 64 if first == 0 else 5000, 9, 1, 0) >= 32768)[:n - first]
        assert torch.equal((y[first:first + keep.numel()] != 0).cpu(), keep)
