"""The cross entropy of a frozen head and its gradient, against the 64-bit form."""

import math

import pytest
import torch

from train_ref import BF16, DEV, F32, ce64, check_ce, rnd, within

pytestmark = pytest.mark.gpu


def problem(M, h, V, seed=0, hide=0.0, spread=2.0, lift=8.0):
    """Rows whose logits have a spread, the label's raised for some; a share of the labels hidden."""
    g = torch.Generator().manual_seed(seed + 100)
    W = rnd(V, h, seed=seed, scale=h ** -0.5)
    labels = torch.randint(0, V, (M,), generator=g).to(DEV)
    x = spread * rnd(M, h, seed=seed + 1, dtype=torch.float32)
    x = (x + lift * torch.rand(M, 1, generator=g).to(DEV) * W[labels].float()).to(torch.bfloat16)
    labels[torch.rand(M, generator=g).to(DEV) < hide] = -100
    return x, W, labels


SIZES = [(1, 8, 1), (1, 8, 2), (2, 16, 15), (3, 64, 17), (5, 72, 255), (7, 64, 256), (31, 128, 257), (64, 128, 300),
         (130, 96, 1000), (127, 256, 4096), (257, 264, 5003), (300, 896, 3001), (513, 128, 40001), (16, 4096, 32000)]


@pytest.mark.parametrize("M,h,V", SIZES)
def test_loss_and_gradient(lib, M, h, V):
    for hide, reduction in ((0.0, "mean"), (0.4, "sum")):
        x, W, y = problem(M, h, V, seed=M, hide=hide)
        got = lib.linear_cross_entropy(x, W, y, reduction=reduction)
        check_ce(got, x, W, y, reduction=reduction)
        alone = lib.linear_cross_entropy(x, W, y, reduction=reduction, grad=False)
        check_ce(alone, x, W, y, reduction=reduction)
        assert alone[3] is None
    assert lib.poll_status() == 0


OPTIONS = [dict(scale=0.25), dict(scale=-1.5), dict(softcap=5.0), dict(softcap=30.0, scale=2.0), dict(smoothing=0.1),
           dict(smoothing=0.9, scale=0.5), dict(softcap=8.0, smoothing=0.2), dict(ignore_index=3)]


@pytest.mark.parametrize("kw", OPTIONS, ids=lambda k: "-".join(f"{a}{b}" for a, b in k.items()))
@pytest.mark.parametrize("M,h,V", [(1, 8, 1), (3, 64, 17), (64, 128, 300), (257, 264, 5003)])
def test_options(lib, M, h, V, kw):
    x, W, y = problem(M, h, V, seed=3)
    if "ignore_index" in kw:
        y[::2] = 3
    got = lib.linear_cross_entropy(x, W, y, **kw)
    check_ce(got, x, W, y, **kw)
    check_ce(lib.linear_cross_entropy(x, W, y, grad=False, **kw), x, W, y, **kw)
    assert lib.poll_status() == 0


@pytest.mark.parametrize("seen", [[], [0], [129], [0, 64, 129], list(range(0, 130, 3))])
@pytest.mark.parametrize("smoothing,softcap", [(0.0, 0.0), (0.1, 0.0), (0.1, 6.0)])
def test_few_or_no_labels(lib, seen, smoothing, softcap):
    """Tokens without a label have no part: zeros, whatever their rows hold.  With none at all the loss
    is 0."""
    x, W, y = problem(130, 64, 700)
    y[[i for i in range(130) if i not in seen]] = -100
    clean = x.clone()
    x[y == -100] = float("nan")
    got = lib.linear_cross_entropy(x, W, y, smoothing=smoothing, softcap=softcap)
    check_ce(got, clean, W, y, smoothing=smoothing, softcap=softcap)
    hidden = y == -100
    assert not bool(got[1][hidden].any()) and not bool(got[2][hidden].any()) and not bool(got[3][hidden].any())
    if not seen:
        assert float(got[0]) == 0.0
    assert lib.poll_status() == 0


def test_labels_outside_the_vocabulary(lib):
    """Reported, and taken as no label."""
    x, W, y = problem(20, 64, 100)
    z = y.clone()
    z[3], z[7], z[11] = 100, -5, 1 << 40
    got = lib.linear_cross_entropy(x, W, z)
    assert lib.poll_status() == 7
    y[[3, 7, 11]] = -100
    want = lib.linear_cross_entropy(x, W, y)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert lib.poll_status() == 0


@pytest.mark.parametrize("gap", [20.0, 90.0, 110.0, 200.0, 3000.0])
@pytest.mark.parametrize("smoothing", [0.0, 0.1])
def test_labels_far_below_the_largest_logit(lib, gap, smoothing):
    """A row's largest logit stands far above its label's: past 100 the piece is taken again."""
    M, h, V = 300, 64, 1000
    x, W, y = problem(M, h, V, spread=1.0, lift=0.0)
    other = (y + 1 + torch.arange(M, device=DEV) % 500) % V
    d = W[other].float() - W[y].float()
    far = x.float() + gap * d / d.square().sum(1, keepdim=True)
    x = torch.where((torch.arange(M, device=DEV) % 7 == 2)[:, None], far, x.float()).to(torch.bfloat16)
    got = lib.linear_cross_entropy(x, W, y, smoothing=smoothing)
    check_ce(got, x, W, y, smoothing=smoothing)
    check_ce(lib.linear_cross_entropy(x, W, y, smoothing=smoothing, grad=False), x, W, y, smoothing=smoothing)
    assert lib.poll_status() == 0


def test_a_label_far_above_all_others(lib):
    """1 - p keeps its precision where p is near 1: the loss and the gradient of sure tokens."""
    M, h, V = 64, 64, 1000
    x, W, y = problem(M, h, V, spread=0.5, lift=0.0)
    w = W[y].float()
    x = (x.float() + torch.linspace(5, 90, M, device=DEV)[:, None] * w / w.square().sum(1, keepdim=True)).to(torch.bfloat16)
    total, loss, lse, dx = lib.linear_cross_entropy(x, W, y, reduction="sum")
    off = ce64(x, W, y, reduction="sum")[4]
    # the others' weights relative to the label's: lse - z_y itself cancels in 64 bits too
    z = x.double() @ W.double().T
    r = torch.exp(z - z.gather(1, y[:, None])).scatter(1, y[:, None], 0.0)
    l64 = torch.log1p(r.sum(1))
    d64 = (r / (1 + r.sum(1, keepdim=True))) @ W.double() - (r.sum(1) / (1 + r.sum(1)))[:, None] * W[y].double()
    # relative to the loss itself: logits are off by `off`, which moves 1 - p by that share of it.  A
    # weight is 2^(z - z_y - 58) in units of ln 2, and one below 2^-126 counts as zero: each of the V
    # terms may lack 2^-68 of the label's, and so may the gradient, times a row of W.
    lost = V * 2.0 ** -68
    within(loss, l64, (2 * off + 100 * F32) * l64 + lost, "loss")
    size = d64.norm(dim=1)
    most = float(W.double().norm(dim=1).max())
    assert bool(((dx.double() - d64).norm(dim=1) <= (4 * BF16 + 4 * off) * size + 2 * lost * most).all())


def test_what_is_not_finite_stays_in_its_row(lib):
    x, W, y = problem(140, 64, 600)
    clean = lib.linear_cross_entropy(x, W, y, reduction="sum")
    bad = x.clone()
    bad[5, 3] = float("nan")
    bad[130, 0] = float("inf")
    total, loss, lse, dx = lib.linear_cross_entropy(bad, W, y, reduction="sum")
    keep = [i for i in range(140) if i not in (5, 130)]
    assert torch.equal(loss[keep], clean[1][keep]) and torch.equal(lse[keep], clean[2][keep])
    assert bool(total.isnan()) and bool(loss[5].isnan()) and not bool(loss[130].isfinite())
    assert bool(dx[5].isnan().all()) and not bool(dx[130].isfinite().all())
    within(dx[keep], clean[3][keep].double(), 2 * BF16 * clean[3][keep].double().abs() + 1e-2 * BF16, "dx")


@pytest.mark.parametrize("grad", [True, False])
def test_pieces(lib, grad):
    """More tokens than a piece holds (a vocabulary of a million: 512 tokens), the last one short or empty."""
    M, h, V = 700, 16, 1_000_003
    for hide in (0.0, 0.9):
        x, W, y = problem(M, h, V, hide=hide)
        total, loss, lse, dx = lib.linear_cross_entropy(x, W, y, grad=grad)
        n = max(1, int((y != -100).sum()))
        for a in range(0, M, 100):                    # 64-bit logits of some tokens at a time
            part = slice(a, a + 100)
            _, l64, s64, d64, off, slack = ce64(x[part], W, y[part], reduction="sum")
            within(loss[part], l64, off + 4 * F32 * l64.abs(), "loss")
            if grad:
                within(dx[part], d64 / n, slack / n, "dx")
        assert abs(float(total) - float(loss.double().sum()) / n) <= 4 * F32 * float(loss.double().sum()) / n


def test_pieces_of_a_small_vocabulary(lib):
    """The product's f32 sums bound the piece: 512 tokens at the widest rows here."""
    M, h, V = 1100, 1 << 19, 24
    g = torch.Generator(device=DEV).manual_seed(3)
    W = (torch.randn(V, h, generator=g, device=DEV) * h ** -0.5).to(torch.bfloat16)
    x = (2 * torch.randn(M, h, generator=g, device=DEV)).to(torch.bfloat16)
    y = torch.randint(0, V, (M,), generator=g, device=DEV)
    y[::9] = -100
    total, loss, lse, dx = lib.linear_cross_entropy(x, W, y)
    n = int((y != -100).sum())
    for part in (slice(0, 40), slice(560, 600), slice(1080, 1100)):
        _, l64, s64, d64, off, slack = ce64(x[part], W, y[part], reduction="sum")
        within(loss[part], l64, off + 4 * F32 * l64.abs(), "loss")
        within(dx[part], d64 / n, slack / n, "dx")
    assert lib.poll_status() == 0


def test_a_head_beyond_32_bit_offsets(lib):
    """2.5G weights: rows far past 2^31 elements, for the logits, the label's row and the gradient."""
    M, h, V = 40, 4096, 600_000
    g = torch.Generator(device=DEV).manual_seed(4)
    W = torch.empty(V, h, dtype=torch.bfloat16, device=DEV)
    for a in range(0, V, 50_000):
        W[a:a + 50_000] = torch.randn(50_000, h, generator=g, device=DEV) * h ** -0.5
    y = torch.randint(0, V, (M,), generator=g, device=DEV)
    y[0], y[1] = V - 1, 0
    x = (torch.randn(M, h, generator=g, device=DEV) + 12 * W[y].float()).to(torch.bfloat16)
    total, loss, lse, dx = lib.linear_cross_entropy(x, W, y, reduction="sum")
    z = torch.cat([x.double() @ W[a:a + 50_000].double().T for a in range(0, V, 50_000)], 1)
    s64 = torch.logsumexp(z, 1)
    # (off as in ce64: 256 + 16 roundings of the running sum of up to |x| |w| in 16-product steps)
    off = 2 * (h / 16 + 16) * 4 * F32 * float((x[:4].double().abs() @ W[:2000].double().abs().T).max()) + 1e-4
    within(lse, s64, off, "lse")
    within(loss, s64 - z.gather(1, y[:, None])[:, 0], off, "loss")
    p = torch.exp(z - s64[:, None]).scatter_add(1, y[:, None], torch.full((M, 1), -1.0, dtype=torch.float64, device=DEV))
    d64 = sum(p[:, a:a + 50_000] @ W[a:a + 50_000].double() for a in range(0, V, 50_000))
    assert float((dx.double() - d64).norm()) <= (2 * BF16 + 2 * off) * float(d64.norm())
    assert lib.poll_status() == 0


def test_same_bits_every_time_and_inside_its_rows(lib):
    x, W, y = problem(200, 128, 3000, hide=0.2)
    a = lib.linear_cross_entropy(x, W, y)
    buf = torch.full((202, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    b = lib.linear_cross_entropy(x, W, y, dx=buf[1:-1])
    assert b[3].data_ptr() == buf[1:-1].data_ptr()
    for p, q in zip(a, b):
        assert torch.equal(p, q)
    assert bool((buf[0] == 7).all()) and bool((buf[-1] == 7).all())


def test_no_tokens(lib):
    W = rnd(50, 64)
    x = torch.empty(0, 64, dtype=torch.bfloat16, device=DEV)
    total, loss, lse, dx = lib.linear_cross_entropy(x, W, torch.empty(0, dtype=torch.int64, device=DEV))
    assert float(total) == 0.0 and loss.shape == (0,) and dx.shape == (0, 64)


def test_in_a_graph_with_other_labels_at_each_replay(lib):
    """How many tokens are labelled is found on the device: a captured call follows it."""
    x, W, y = problem(300, 128, 2000)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        lib.linear_cross_entropy(x, W, y)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            got = lib.linear_cross_entropy(x, W, y)
    for hide in (0.0, 0.95, 1.0, 0.5):
        torch.cuda.synchronize()
        a, _, b = problem(300, 128, 2000, seed=int(10 * hide), hide=hide)
        x.copy_(a)
        y.copy_(b)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for p, q in zip(got, lib.linear_cross_entropy(x, W, y)):
            assert torch.equal(p, q)
    assert lib.poll_status() == 0


def test_two_streams_at_once(lib):
    work = [problem(500, 128, 9001, seed=i) for i in range(2)]
    want = [lib.linear_cross_entropy(*w) for w in work]
    streams = [torch.cuda.Stream() for _ in work]
    torch.cuda.synchronize()
    got = []
    for _ in range(3):
        for s, w in zip(streams, work):
            with torch.cuda.stream(s):
                got.append(lib.linear_cross_entropy(*w))
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(g, want[i % 2]))


@pytest.mark.parametrize("M,h", [(0, 64), (1, 8), (7, 72), (300, 896), (5000, 4096)])
def test_scaled_rows(lib, M, h):
    x, g = rnd(M, h), rnd(M, seed=1, dtype=torch.float32)
    for f in (g, g.sum() + 1.5):
        want = x.double() * (f.double()[:, None] if f.dim() else f.double())
        within(lib.scale_rows(x, f), want, BF16 * want.abs() + 1e-40)
    y = x.clone()
    assert lib.scale_rows(y, g, out=y) is y and torch.equal(y, lib.scale_rows(x, g))
    assert torch.equal(lib.scale_rows(x, torch.ones((), device=DEV)), x)


@pytest.mark.parametrize("reduction", ["mean", "sum", "none"])
def test_autograd(lib, reduction):
    from rank_mlp_gb300.autograd import lora_linear_cross_entropy
    x, W, y = problem(60, 64, 500, hide=0.3)
    x, y = x.view(3, 20, 64).requires_grad_(), y.view(3, 20)
    loss = lora_linear_cross_entropy(x, W, y, softcap=20.0, reduction=reduction)
    total, each, _, dx = lib.linear_cross_entropy(x.detach().view(60, 64), W, y.reshape(-1), softcap=20.0,
                                                  reduction="sum" if reduction == "none" else reduction)
    if reduction == "none":
        assert torch.equal(loss.detach().view(-1), each)
        g = rnd(3, 20, seed=7, dtype=torch.float32)
        loss.backward(g)
        within(x.grad.view(60, 64), dx.double() * g.view(60, 1).double(), BF16 * (dx.double() * g.view(60, 1)).abs())
    else:
        assert torch.equal(loss.detach(), total)
        loss.backward()
        assert torch.equal(x.grad.view(60, 64), dx)
        x.grad = None
        (8.0 * lora_linear_cross_entropy(x, W, y, softcap=20.0, reduction=reduction)).backward()
        assert torch.equal(x.grad.view(60, 64), 8 * dx)
    # against differences of the 64-bit loss along a direction
    d = rnd(60, 64, seed=9).double()
    kw = dict(softcap=20.0, reduction="sum")
    f = lambda t: float(ce64(x.detach().view(60, 64).double() + t * d, W, y.reshape(-1), **kw)[0])  # noqa: E731
    want = (f(1e-4) - f(-1e-4)) / 2e-4
    dsum = lib.linear_cross_entropy(x.detach().view(60, 64), W, y.reshape(-1), **kw)[3].double()
    slack = ce64(x.detach().view(60, 64), W, y.reshape(-1), **kw)[5]
    assert abs(float((dsum * d).sum()) - want) <= float((slack * d.abs()).sum()) + 1e-4 * abs(want)
    with torch.no_grad():
        assert lora_linear_cross_entropy(x, W, y).grad_fn is None
    assert lib.poll_status() == 0


def test_a_wait_that_runs_out_is_reported_and_the_next_call_is_right(lib):
    x, W, y = problem(300, 128, 2000)
    want = lib.linear_cross_entropy(x, W, y)
    torch.cuda.synchronize()
    for grad in (True, False):
        try:
            lib.set_wait_timeout(20_000_000)
            lib.test_expire_waits(1)
            lib.linear_cross_entropy(x, W, y, grad=grad)
            torch.cuda.synchronize()
            assert lib.poll_status() == 6
        finally:
            lib.test_expire_waits(0)
            lib.set_wait_timeout(0)
    assert math.isfinite(float(want[0]))
    for a, b in zip(want, lib.linear_cross_entropy(x, W, y)):
        assert torch.equal(a, b)
    assert lib.poll_status() == 0
