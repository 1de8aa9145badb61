"""Rows whose logits are summed in parts: lengths about the parts' ends, every option, the second try, a wait that
runs out."""

import pytest
import torch

from train_ref import DEV, check_ce, rnd

pytestmark = pytest.mark.gpu


def problem(M, h, V, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    W = (torch.randn(V, h, generator=g, device=DEV) * h ** -0.5).to(torch.bfloat16)
    y = torch.randint(0, V, (M,), generator=g, device=DEV)
    x = (2 * torch.randn(M, h, generator=g, device=DEV) + 8 * torch.rand(M, 1, generator=g, device=DEV) * W[y].float()).to(torch.bfloat16)
    y[torch.rand(M, generator=g, device=DEV) < 0.2] = -100
    return x, W, y


@pytest.mark.parametrize("M,V", [(1, 3), (70, 700), (300, 5003)])
@pytest.mark.parametrize("h", [1016, 1024, 1032, 1080, 1088, 2048, 2056, 2064, 4104, 5000])
def test_lengths(lib, h, M, V):
    x, W, y = problem(M, h, V, seed=h + M)
    if M == 1:
        y[:] = 2
    for kw in (dict(), dict(reduction="sum", smoothing=0.1), dict(softcap=6.0), dict(softcap=20.0, smoothing=0.2, scale=0.5)):
        check_ce(lib.linear_cross_entropy(x, W, y, **kw), x, W, y, **kw)
        check_ce(lib.linear_cross_entropy(x, W, y, grad=False, **kw), x, W, y, **kw)
    assert lib.poll_status() == 0


@pytest.mark.parametrize("softcap", [0.0, 400.0])
def test_a_piece_that_is_taken_again(lib, softcap):
    M, h, V = 300, 2056, 1000
    x, W, y = problem(M, h, V)
    y = torch.where(y == -100, 5, y)
    far = W[(y + 7) % V].float() - W[y].float()
    x = torch.where((torch.arange(M, device=DEV) % 50 == 3)[:, None], x.float() + 130 * far / far.square().sum(1, keepdim=True), x.float()).to(torch.bfloat16)
    z = x.double() @ W.double().T
    assert float((z.amax(1) - z.gather(1, y[:, None])[:, 0]).max()) > 110
    check_ce(lib.linear_cross_entropy(x, W, y, softcap=softcap), x, W, y, softcap=softcap)
    assert lib.poll_status() == 0


def test_tokens_do_not_depend_on_their_place(lib):
    """The same row in any tile, beside any others: the same loss and lse, bit for bit."""
    x, W, y = problem(700, 2056, 1003)
    y = torch.where(y == -100, 5, y)
    _, loss, lse, _ = lib.linear_cross_entropy(x, W, y, reduction="sum")
    turn = torch.randperm(700, device=DEV)
    _, l, s, _ = lib.linear_cross_entropy(x[turn], W, y[turn], reduction="sum")
    assert torch.equal(loss[turn], l) and torch.equal(lse[turn], s)
    _, l, s, _ = lib.linear_cross_entropy(x[333:334], W, y[333:334], reduction="sum")
    assert torch.equal(loss[333:334], l) and torch.equal(lse[333:334], s)


def test_a_wait_that_runs_out_is_reported_and_the_next_call_is_right(lib):
    x, W, y = problem(600, 2056, 3000)
    want = {grad: lib.linear_cross_entropy(x, W, y, grad=grad) for grad in (True, False)}
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
        for a, b in zip(want[grad], lib.linear_cross_entropy(x, W, y, grad=grad)):
            assert a is b is None or torch.equal(a, b)
    assert lib.poll_status() == 0


@pytest.mark.parametrize("far", [[5], [990], [5, 990]])
def test_pieces_of_which_some_are_taken_again(lib, far):
    """Two pieces of tokens; the total waits for the last one's second try."""
    from train_ref import F32, ce64, within
    M, h, V = 1000, 24, 600_011
    x, W, y = problem(M, h, V, seed=3)
    y[far] = 17
    d = W[400_000].float() - W[17].float()
    x[far] = (x[far].float() + 150 * d / d.square().sum()).to(torch.bfloat16)
    total, loss, lse, dx = lib.linear_cross_entropy(x, W, y)
    n = int((y != -100).sum())
    for a in (0, 460, 940):
        part = slice(a, a + 60)
        _, l64, s64, d64, off, slack = ce64(x[part], W, y[part], reduction="sum")
        within(loss[part], l64, off + 4 * F32 * l64.abs(), "loss")
        within(lse[part], s64, off + 4 * F32 * s64.abs(), "lse")
        within(dx[part], d64 / n, slack / n, "dx")
    want = float(loss.double().sum()) / n
    assert abs(float(total) - want) <= 4 * F32 * want and float(loss[far].min()) > 100
    assert lib.poll_status() == 0
